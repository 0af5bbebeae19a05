// gemm_fp4_kernel.cuh -- D = alpha * A * B^T of microscaled 4-bit matrices on the
// tensor cores (tcgen05.mma kind::mxf4 and kind::mxf4nvf4, block_scale).
//
// Data path: A, B -TMA-> 128-byte swizzled SMEM -tcgen05.mma-> TMEM (fp32); the
// scale tiles (512 bytes: 128 rows x 4 blocks, stored in global memory in the
// order the tensor cores take them) -TMA-> SMEM -tcgen05.cp-> TMEM, where the
// MMA reads them.  The products and their scales are exact in fp32; the sum is
// fp32, multiplied by alpha (and before it, exactly, by a power of two where alpha
// alone would leave fp32's range) and rounded once.
//
// A stage is a K tile of 256 elements: 128 bytes of each row, four MMAs of
// K = 64.  Scale tiles of a stage: two (FP4_MX: 8 blocks of 32, 2 scales per
// MMA and row) or four (FP4_NV: 16 blocks of 16, 4 per MMA and row).  Past the
// ends of A, B and the scales TMA fills zeros, so every stage is whole: its
// zero codes add nothing.
#pragma once

#include "../gemm_kernel.cuh"
#include "common.cuh"
#include "fp4.cuh"

namespace linear_ops {

using gemm_f16::PipelineState;
using gemm_f16::wait_bounded;
using gemm_f16::WorkItem;

namespace ptx4 {

// 3-D tiled loads (scale tiles), into this CTA's shared memory; the second form
// may signal the barrier of the pair's leader.
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

// An arrival, possibly on the peer's barrier, that publishes no memory writes: a
// release at cluster scope would first wait for all of the thread's.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// Shared-memory descriptor of one scale tile: no swizzle, 8 x 16-byte core
// matrices 128 bytes apart (fields as in ptx::smem_desc_k_sw128).
__device__ __forceinline__ uint64_t scale_desc(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(128u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    return d;
}

// One scale tile (32 rows of 16 bytes) into 4 TMEM columns, repeated in each of
// the four 32-lane quarters.  Ordered with the MMAs that this thread issues.
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (CG == 2) {
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    } else {
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    }
}

// D(tmem) (+)= (A * its scales) * (B * its scales)^T over K = 64.
template <int CG, bool NV>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                        uint32_t accumulate) {
#define LINEAR_MMA_FP4(GROUP, KIND, VECS)                                                                         \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                \
                 "tcgen05.mma.cta_group::" GROUP ".kind::" KIND ".block_scale.scale_vec::" VECS                   \
                 " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                               \
                 "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)                                    \
                 : "memory")
    if constexpr (CG == 2 && NV) {
        LINEAR_MMA_FP4("2", "mxf4nvf4", "4X");
    } else if constexpr (CG == 2) {
        LINEAR_MMA_FP4("2", "mxf4", "2X");
    } else if constexpr (NV) {
        LINEAR_MMA_FP4("1", "mxf4nvf4", "4X");
    } else {
        LINEAR_MMA_FP4("1", "mxf4", "2X");
    }
#undef LINEAR_MMA_FP4
}

}  // namespace ptx4

// Instruction descriptor of the block-scaled 4-bit MMAs (PTX ISA): A and B E2M1
// [7,10)=[10,12)=1, both K-major, N>>3 at [17,23), scale type at 23 (0 E4M3,
// 1 E8M0), M>>7 at [27,29), K = 64 at 31; [4,6) and [29,31) say at which byte of
// a column's word the scales of B and A start (0, or 2 for the second pair).
__host__ __device__ constexpr uint32_t idesc_fp4(int M, int N, bool nv, uint32_t scale_byte) {
    return (scale_byte << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | ((nv ? 0u : 1u) << 23) |
           (static_cast<uint32_t>(M >> 7) << 27) | (scale_byte << 29);
}

// What both kernels share about a stage.  CG: CTAs of a tile, BN: rows of B per
// tile.  A CTA holds 128 rows of A and BN / CG of B, but the scales of all BN.
template <int CG, int BN, bool NV>
struct Fp4Stage {
    static constexpr int BLOCK_K = 256;                       // elements: 128 bytes of a row
    static constexpr int SF_TILES = NV ? 4 : 2;               // scale tiles of 128 rows
    static constexpr int SFB_ROWS = BN > 128 ? BN / 128 : 1;  // row tiles of B's scales
    static constexpr int A_BYTES = 128 * 128;
    static constexpr int B_BYTES = BN / CG * 128;
    static constexpr int SFA_BYTES = SF_TILES * kScaleTileBytes;
    static constexpr int SFB_BYTES = SFB_ROWS * SF_TILES * kScaleTileBytes;
    static constexpr int BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
    static constexpr uint32_t TX = BYTES * CG;
    static constexpr int SFA_COLS = SF_TILES * 4;             // TMEM columns of a stage's scales
    static constexpr int SFB_COLS = SF_TILES * 4 * SFB_ROWS;
    static constexpr int SF_COLS = SFA_COLS + SFB_COLS;
    static_assert(A_BYTES % 1024 == 0 && B_BYTES % 1024 == 0, "1 KiB swizzle atoms");

    // The copies of a stage's scales to TMEM columns `tsf`, in order with the MMAs
    // issued before and after them.
    static __device__ __forceinline__ void copy_scales(uint32_t ssfa, uint32_t ssfb, uint32_t tsf) {
        const uint32_t tsfa = tsf, tsfb = tsf + SFA_COLS;
#pragma unroll
        for (int j = 0; j < SF_TILES; ++j) {
            ptx4::copy_scales<CG>(tsfa + 4 * j, ptx4::scale_desc(ssfa + j * kScaleTileBytes));
#pragma unroll
            for (int r = 0; r < SFB_ROWS; ++r) {
                ptx4::copy_scales<CG>(tsfb + (j * SFB_ROWS + r) * 4,
                                      ptx4::scale_desc(ssfb + (r * SF_TILES + j) * kScaleTileBytes));
            }
        }
    }
    // A stage's four MMAs.  B's rows start on a scale tile: the MMA takes its scales
    // from a multiple of 4 columns on (an odd column is a misaligned address), so not
    // from a tile's middle.
    static __device__ __forceinline__ void multiply(uint32_t sa, uint32_t sb, uint32_t tsf, uint32_t d, bool first) {
        const uint32_t tsfa = tsf, tsfb = tsf + SFA_COLS;
        const uint64_t a_desc = ptx::smem_desc_k_sw128(sa), b_desc = ptx::smem_desc_k_sw128(sb);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = NV ? k : k / 2;  // its scale tile
            const uint64_t koff = static_cast<uint64_t>(k * 32 / 16);
            constexpr uint32_t even = idesc_fp4(128 * CG, BN, NV, 0), odd = idesc_fp4(128 * CG, BN, NV, 2);
            ptx4::mma_fp4<CG, NV>(d, a_desc + koff, b_desc + koff, !NV && k % 2 ? odd : even, tsfa + 4 * j,
                                  tsfb + 4 * SFB_ROWS * j, first && k == 0 ? 0u : 1u);
        }
    }
};

struct Fp4Params {
    int32_t M, N;                  // of D
    int32_t m_tiles, n_tiles;      // of the tile's 128- (256-) row side and of its other side
    int32_t k_tiles;
    int32_t raster_group;
    int32_t d_type;
    int32_t swap;                  // single-CTA tiles: the 128-row side is B
    int32_t tma_store;             // CTA pairs: D through its tensor map
    int32_t wide_store;            // single-CTA tiles: D's rows are aligned units of four elements
    uint32_t debug_flags;
    uint64_t timeout_ns;
    float first, alpha;            // D = (sum * first) * alpha; first is a power of two
    void *D;
};

__device__ __forceinline__ void store_d(void *D, int32_t type, int64_t at, float v) {
    if (type == LINEAR_F16) {
        static_cast<__half *>(D)[at] = __float2half_rn(v);
    } else if (type == LINEAR_BF16) {
        static_cast<__nv_bfloat16 *>(D)[at] = __float2bfloat16_rn(v);
    } else {
        static_cast<float *>(D)[at] = v;
    }
}

__device__ __forceinline__ uint32_t pack16(int32_t type, float lo, float hi) {
    if (type == LINEAR_F16) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Four consecutive elements of a row of D, of which `left` are in the row.
__device__ __forceinline__ void store_d4(const Fp4Params &p, int64_t at, int32_t left, float4 v) {
    if (p.wide_store) {  // rows of whole units of four, aligned
        if (p.d_type == LINEAR_F32) {
            *reinterpret_cast<float4 *>(static_cast<float *>(p.D) + at) = v;
        } else {
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.D) + at) =
                make_uint2(pack16(p.d_type, v.x, v.y), pack16(p.d_type, v.z, v.w));
        }
        return;
    }
    store_d(p.D, p.d_type, at, v.x);
    if (left > 1) store_d(p.D, p.d_type, at + 1, v.y);
    if (left > 2) store_d(p.D, p.d_type, at + 2, v.z);
    if (left > 3) store_d(p.D, p.d_type, at + 3, v.w);
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[N]) {
    if constexpr (N == 32) {
        ptx::tmem_ld_32x32b_x32(taddr, v);
    } else {
        ptx::tmem_ld_32x32b_x16(taddr, v);
    }
}

// Two sums times first, exactly, and alpha.  Packed, the two multiplications take as
// many instructions as one by itself did (1000 x 1529 x 2088 8.3 us either way; with a
// branch around the first one 8.4).
__device__ __forceinline__ float2 scaled(const Fp4Params &p, uint32_t a, uint32_t b) {
    return mul2(mul2(make_float2(__uint_as_float(a), __uint_as_float(b)), both(p.first)), both(p.alpha));
}
__device__ __forceinline__ uint32_t scaled16(const Fp4Params &p, uint32_t a, uint32_t b) {
    const float2 v = scaled(p, a, b);
    return pack16(p.d_type, v.x, v.y);
}

// Four sums of a CTA of the cluster (of this CTA without a K split).
template <int KS>
__device__ __forceinline__ float4 load_sums(uint32_t addr) {
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

// ------------------------------------------------------- single-CTA tiles --
//
// One CTA of 6 warps per tile and K slice (warp 0 TMA producer, warp 1 MMA
// issuer and TMEM allocator, warps 2-5 read the accumulator).  The 128-row side
// is called P, the other Q (BN rows): without swap P is A, with it P is B,
// which for few rows of A streams the weights through the 128-row side.  Tiles
// of BN < 128 are for a Q of at most BN rows (see Fp4Stage::multiply).  KS
// CTAs of a cluster share a tile's K; their fp32 sums meet through distributed
// shared memory, added in slice order, rounded once.
//
// For few rows of Q the time is P's bytes: 1 x 8192 x 8192 mx 7.8 us, 4.6 TB/s (5.3
// us at the copy rate; launch, first loads, the cluster's sums and the end take the
// rest), 64 x 28672 x 4096 nv 13.8 us, 5.1 TB/s.  D's rows of whole units of four go
// in one store for each; others element by element: 64 x 4096 x 4096 mx 5.6 us, 64 x
// 4097 x 4096 6.0.
template <int BN, int KS, bool NV>
struct Fp4Single {
    using S = Fp4Stage<1, BN, NV>;
    // two CTAs an SM, so that one's start and end pass under the other's loads: half of
    // 228 KiB, less 1 KiB that each takes beside its own
    static constexpr int BUDGET = 113 * 1024;
    static constexpr int REST = 8 + 16 + 896;  // barrier, flags, from a multiple of 128 bytes to one of 1024
    static constexpr int STAGES = (BUDGET - REST) / (S::BYTES + 16);
    static constexpr int SF_BUFS = 2;
    static constexpr int OFF_A = 0;
    static constexpr int OFF_B = OFF_A + STAGES * S::A_BYTES;
    static constexpr int OFF_SFA = OFF_B + STAGES * S::B_BYTES;
    static constexpr int OFF_SFB = OFF_SFA + STAGES * S::SFA_BYTES;
    static constexpr int RING = OFF_SFB + STAGES * S::SFB_BYTES;
    // The CTA's fp32 sums, in the ring once it is idle, in the order of D's rows: with
    // swap row q of Q (128 sums) at q * LD_SWAP, else row p of P (BN sums) at p * LD.
    // Rows are 16 bytes off a multiple of 128 bytes, so the 16-byte accesses of 8
    // lanes in 8 rows meet no bank twice.
    static constexpr int LD = BN + 4, LD_SWAP = 128 + 4;
    static constexpr int SUMS = 4 * (128 * LD > BN * LD_SWAP ? 128 * LD : BN * LD_SWAP);
    static constexpr int OFF_BAR = RING > SUMS ? RING : (SUMS + 15) / 16 * 16;
    static constexpr int OFF_MISC = OFF_BAR + (2 * STAGES + 1) * 8;
    static constexpr int SMEM_ALLOC = OFF_MISC + 16 + 896;
    static constexpr int TMEM_USED = BN + SF_BUFS * S::SF_COLS;
    static constexpr int TMEM_COLS = TMEM_USED <= 64 ? 64 : (TMEM_USED <= 128 ? 128 : 256);
    static constexpr int SF_COL = BN;
    static constexpr int THREADS = 192;
    static_assert(TMEM_USED <= 256 && STAGES >= 3 && SMEM_ALLOC <= BUDGET, "two CTAs an SM");
    static_assert(BN == 16 || BN == 32 || BN == 64 || BN == 128, "tile width");
};

template <int BN, int KS, bool NV>
__global__ void __launch_bounds__(192, 2)
    fp4_single_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmSP, const __grid_constant__ CUtensorMap tmSQ,
                      const Fp4Params p) {
    using C = Fp4Single<BN, KS, NV>;
    using S = typename C::S;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
    const int lane = static_cast<int>(threadIdx.x) % 32;

    const uint32_t bar_full = base + C::OFF_BAR, bar_empty = bar_full + 8 * C::STAGES;
    const uint32_t bar_done = bar_empty + 8 * C::STAGES;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);

    // the tile and K slice of this CTA
    const int rank = KS > 1 ? static_cast<int>(blockIdx.x) % KS : 0;
    const int tile = static_cast<int>(blockIdx.x) / KS;
    const int pt = tile / p.n_tiles, qt = tile % p.n_tiles;
    const int kt_begin = static_cast<int>(static_cast<int64_t>(p.k_tiles) * rank / KS);
    const int kt_end = static_cast<int>(static_cast<int64_t>(p.k_tiles) * (rank + 1) / KS);
    const int p0 = pt * 128, q0 = qt * BN;

    if (warp == 0 && lane == 0) {
        ptx::prefetch_tensormap(&tmP);
        ptx::prefetch_tensormap(&tmQ);
        ptx::prefetch_tensormap(&tmSP);
        ptx::prefetch_tensormap(&tmSQ);
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
    ptx::tcgen05_fence_before();
    __syncthreads();
    ptx::tcgen05_fence_after();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();

    if (warp == 0) {
        if (ptx::elect_one()) {
            // L2 is told of the first ring fill before the wait for the previous
            // kernel (a hint: it changes no value)
            for (int kt = kt_begin; kt < kt_end && kt < kt_begin + C::STAGES; ++kt) {
                ptx::tma_prefetch_l2_2d(&tmP, kt * 128, p0);
            }
            ptx::griddep_wait();
            PipelineState ring(C::STAGES, (p.debug_flags & 1u) ? 0u : 1u);
            bool ok = true;
            for (int kt = kt_begin; kt < kt_end; ++kt) {
                if (!wait_bounded(bar_empty + 8 * ring.stage, ring.phase, abort_flag, p.timeout_ns,
                                  gemm_f16::kRoleProducer, kt)) {
                    ok = false;
                    break;
                }
                const uint32_t full = bar_full + 8 * ring.stage;
                ptx::mbar_arrive_expect_tx(full, S::TX);
                ptx::tma_load_2d(base + C::OFF_A + ring.stage * S::A_BYTES, &tmP, full, kt * 128, p0);
                ptx::tma_load_2d(base + C::OFF_B + ring.stage * S::B_BYTES, &tmQ, full, kt * 128, q0);
                ptx4::tma_load_3d(base + C::OFF_SFA + ring.stage * S::SFA_BYTES, &tmSP, full, 0, kt * S::SF_TILES, pt);
                ptx4::tma_load_3d(base + C::OFF_SFB + ring.stage * S::SFB_BYTES, &tmSQ, full, 0, kt * S::SF_TILES,
                                  q0 / 128);
                ring.advance();
            }
            if (!ok) {  // time for loads in flight to land before the shared memory goes
                const uint64_t t0 = ptx::globaltimer_ns();
                while (ptx::globaltimer_ns() - t0 < 20000) ptx::nanosleep(1000);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (ptx::elect_one()) {
            PipelineState ring(C::STAGES, 0u);
            for (int kt = kt_begin; kt < kt_end; ++kt) {
                if (!wait_bounded(bar_full + 8 * ring.stage, ring.phase, abort_flag, p.timeout_ns, gemm_f16::kRoleMma,
                                  kt)) {
                    break;
                }
                ptx::tcgen05_fence_after();
                const int s = ring.stage;
                const uint32_t tsf = tmem_base + C::SF_COL + (kt - kt_begin) % C::SF_BUFS * S::SF_COLS;
                S::copy_scales(base + C::OFF_SFA + s * S::SFA_BYTES, base + C::OFF_SFB + s * S::SFB_BYTES, tsf);
                S::multiply(base + C::OFF_A + s * S::A_BYTES, base + C::OFF_B + s * S::B_BYTES, tsf, tmem_base,
                            kt == kt_begin);
                ptx::mma_commit<1>(bar_empty + 8 * s, 0x1);
                ring.advance();
            }
            // every MMA issued so far (after an abort as well: TMEM is freed below)
            ptx::mma_commit<1>(bar_done, 0x1);
            wait_bounded(bar_done, 0, abort_flag, p.timeout_ns, gemm_f16::kRoleMma, 0xFFFFFFFFu, false);
        }
        __syncwarp();
    } else {
        // all MMAs done: the accumulator is complete and the ring idle
        bool ok = true;
        if (lane == 0) {
            ok = wait_bounded(bar_done, 0, abort_flag, p.timeout_ns, gemm_f16::kRoleEpilogue, 0);
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (ok && *abort_flag == 0) {
            ptx::tcgen05_fence_after();
            const int row = (warp & 3) * 32 + lane;  // of P
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            constexpr int kCols = BN < 32 ? 16 : 32;  // of a TMEM load
#pragma unroll
            for (int c = 0; c < BN; c += kCols) {
                uint32_t v[kCols];
                tmem_ld<kCols>(taddr + c, v);
                ptx::tmem_wait_ld();
                if (p.first != 1.f) {  // here, not with alpha below, where it costs 64 x 28672 x 4096 nv 0.3 us
#pragma unroll
                    for (int j = 0; j < kCols; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * p.first);
                }
                if (p.swap) {
#pragma unroll
                    for (int j = 0; j < kCols; ++j) {
                        reinterpret_cast<float *>(smem)[(c + j) * C::LD_SWAP + row] = __uint_as_float(v[j]);
                    }
                } else {
                    const uint32_t at = base + static_cast<uint32_t>(row * C::LD + c) * 4u;
#pragma unroll
                    for (int j = 0; j < kCols; j += 4) ptx::st_shared_v4(at + j * 4u, v[j], v[j + 1], v[j + 2], v[j + 3]);
                }
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
    ptx::griddep_wait();
    if (*abort_flag == 0) {
        // Rows of D that this CTA adds up: with swap its share of Q's rows that
        // exist, else of P's; four columns a thread and step.
        const int d_rows = p.swap ? (p.M - q0 < BN ? p.M - q0 : BN) : (p.M - p0 < 128 ? p.M - p0 : 128);
        const int first = d_rows * rank / KS, last = d_rows * (rank + 1) / KS;
        const int per = p.swap ? 32 : BN / 4, ld = p.swap ? C::LD_SWAP : C::LD;  // threads and floats of a row
        const int m0 = p.swap ? q0 : p0, n0 = p.swap ? p0 : q0;
        uint32_t peer[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) peer[s] = KS > 1 ? ptx::mapa(base, static_cast<uint32_t>(s)) : base;
        for (int u = first * per + static_cast<int>(threadIdx.x); u < last * per; u += C::THREADS) {
            const int r = u / per, c = u % per * 4;
            const int32_t n = n0 + c;
            if (n >= p.N) continue;
            const uint32_t at = static_cast<uint32_t>(r * ld + c) * 4u;
            float4 part[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) part[s] = load_sums<KS>(peer[s] + at);
            float4 v = part[0];
#pragma unroll
            for (int s = 1; s < KS; ++s) v.x += part[s].x, v.y += part[s].y, v.z += part[s].z, v.w += part[s].w;
            v.x *= p.alpha, v.y *= p.alpha, v.z *= p.alpha, v.w *= p.alpha;
            store_d4(p, static_cast<int64_t>(m0 + r) * p.N + n, p.N - n, v);
        }
    }
    if constexpr (KS > 1) {
        // no CTA leaves while another reads its sums (they are in registers by now; the
        // arrival need not wait for this thread's stores to D, as a release would)
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

// --------------------------------------------------------------- CTA pairs --
//
// Persistent pairs with 256 x 256 tiles, MMAs of M = 256, N = 256 (roles and
// rings as in gemm_kernel.cuh).  Two 256-column accumulators and two buffers of
// a stage's scales do not fit 512 columns of TMEM, so the accumulators overlap
// in OVER columns: tile i is at columns [0, 256) (i even) or [256 - OVER,
// 512 - OVER).  The epilogue reads the columns that the next tile's accumulator
// shares first and hands them over; all others of that accumulator it has read
// by then, with the tile before.  So the next tile's MMAs wait for OVER columns
// only, and run while the epilogue reads the rest.
//
// Bound by the MMAs, 512 cycles a stage (520 measured, and some 2000 a tile between
// tiles): 8192 x 8192 x 8192 mx 148 us, 7.4 PFLOP/s; 8192 x 28672 x 4096 mx 270 us,
// 7.1, in a short run (300 in a stream of calls under the power cap; nv 300 to 319).  One tile a pair is bound by the start, the first loads and the epilogue:
// 1000 x 1528 x 256 4.5 us, 512 x 4096 x 4096 8.65.  Eight epilogue warps of 128
// columns, as one warp's way through TMEM, registers and staging is latency: with
// four of 256 columns these took 5.0 and 9.2 us.
template <bool NV>
struct Fp4Pair {
    using S = Fp4Stage<2, 256, NV>;
    static constexpr int STAGES = 5;
    static constexpr int SF_BUFS = 2;
    static constexpr int SF_COL = 512 - SF_BUFS * S::SF_COLS;
    static constexpr int OVER = (512 - SF_COL + 31) / 32 * 32;  // 64 (FP4_MX) or 96
    static constexpr int ACC1 = 256 - OVER;                     // second accumulator's first column
    static constexpr int OFF_A = 0;
    static constexpr int OFF_B = OFF_A + STAGES * S::A_BYTES;
    static constexpr int OFF_D = OFF_B + STAGES * S::B_BYTES;
    static constexpr int EPI_WARPS = 8;                         // two for each quarter of the rows, 128 columns each
    static constexpr int EPI_BUF = 32 * 128;                    // of a warp: 32 rows of 128 bytes
    static constexpr int ROW_PITCH = 64 * 2 + 16;               // a row of 64 elements, shifted up to 7
    static constexpr int EPI_ROWS = 32 * ROW_PITCH;             // 32 such rows (the same memory as the buffers)
    static_assert(EPI_ROWS >= EPI_BUF && OFF_D % 1024 == 0 && EPI_WARPS * EPI_ROWS % 1024 == 0, "staging");
    static constexpr int OFF_SFA = OFF_D + EPI_WARPS * EPI_ROWS;
    static constexpr int OFF_SFB = OFF_SFA + STAGES * S::SFA_BYTES;
    static constexpr int OFF_BAR = OFF_SFB + STAGES * S::SFB_BYTES;
    static constexpr int OFF_MISC = OFF_BAR + (2 * STAGES + 4) * 8;
    static constexpr int SMEM_ALLOC = OFF_MISC + 16 + 896;      // from a multiple of 128 bytes to one of 1024
    static constexpr int THREADS = 64 + EPI_WARPS * 32;
    static_assert(ACC1 + 256 <= SF_COL && SMEM_ALLOC <= 232448, "TMEM columns, 227 KiB");
};

// Half HALF (64 columns) of a warp's 32 rows x 128 16-bit elements, a row a lane
// (packed in w; `before`: the row's two elements before them), to rows of D that
// start anywhere; the two halves one after the other.  A lane stages its row with
// the shift that its address has within 16 bytes, so the row's whole units are
// aligned in both memories, and 8 lanes move the units of a row.  The unit that
// the halves share stays in the staging between them; the one that the tile's two
// warps share is moved by the left one, which reads the next eight columns too
// (`after`).  What the tile's first and last unit hold of the row goes in aligned
// words of 8, 4 and 2 bytes.
//
// Rows 8 apart have one shift and, at a pitch of 9 units, the same banks; so the words
// of a unit are rotated by row / 8 in the staging, which who reads whole units undoes
// at compile time.  Two warps run on each scheduler here and little hides their
// latencies, so index arithmetic and accesses count: 1000 x 1529 x 256 takes 5.4 us
// (4.5 at 1528 columns, by TMA), 7252 x 2575 x 405 16.4 (12.4 at 2576); without the
// rotation 5.9 and 17.7, in words of 4 bytes row by row 5.5 and 19.5.
template <int HALF, int PITCH>
__device__ __forceinline__ void store_unaligned(const Fp4Params &p, uint8_t *staging, const uint32_t (&w)[32],
                                                uint32_t before, const uint32_t (&after)[4], bool left, int lane,
                                                int32_t row0, int32_t col0) {
    uint16_t *first = static_cast<uint16_t *>(p.D) + static_cast<int64_t>(row0) * p.N + col0;  // row 0, the slice's start
    const int cols = p.N - col0 > HALF * 64 ? p.N - col0 - HALF * 64 : 0;  // of the row from this half on
    uint8_t *own = staging + lane * PITCH;
    const int turn = lane / 8;
    auto place = [&](int word) {  // in the lane's row
        return reinterpret_cast<uint32_t *>(own) + (word / 4 * 4 + ((word + turn) & 3));
    };
    const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(first + static_cast<int64_t>(lane) * p.N) / 2) & 7);
    if (HALF == 1) {  // the shared unit: last of the first half, first of this one
        *reinterpret_cast<uint4 *>(own) = *reinterpret_cast<const uint4 *>(own + 128);
    }
    const uint32_t odd = static_cast<uint32_t>(shift & 1) * 16u;
    uint32_t *at[4];  // of words 0 to 3; those four further on are a unit further
#pragma unroll
    for (int j = 0; j < 4; ++j) at[j] = place(shift / 2 + j);
#pragma unroll
    for (int k = 0; k < 32; ++k) at[k % 4][k / 4 * 4] = __funnelshift_l(k ? w[k - 1] : before, w[k], odd);
    if (HALF == 1 && left) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // up to the end of the unit
            if (k + shift / 2 < 4) at[k][32] = __funnelshift_l(k ? after[k - 1] : w[31], after[k], odd);
        }
    } else {
        at[0][32] = __funnelshift_l(w[31], 0u, odd);
    }
    __syncwarp();
    {
        // lane: unit lane % 8 of rows lane / 8, 4 + lane / 8, ...
        uint16_t *row = first + HALF * 64 + static_cast<int64_t>(lane >> 3) * p.N;
        const int unit = lane & 7;
        const uint8_t *from = staging + (lane >> 3) * PITCH + unit * 16;
        const int rows = p.M - row0 - (lane >> 3);
        const int64_t four = 4 * static_cast<int64_t>(p.N);
#pragma unroll
        for (int i = 0; i < 8; ++i, row += four) {
            const int s = static_cast<int>(reinterpret_cast<uintptr_t>(row) / 2 & 7);
            // the first half's first unit is whole without a shift, the second's always
            if (4 * i < rows && unit * 8 + 8 <= s + cols && (HALF == 1 || s == 0 || unit > 0)) {
                const uint4 v = *reinterpret_cast<const uint4 *>(from + i * 4 * PITCH);
                const uint32_t t[4] = {v.x, v.y, v.z, v.w};
                const int g = i / 2;  // the row's turn
                *reinterpret_cast<uint4 *>(row + (unit * 8 - s)) =
                    make_uint4(t[g], t[(1 + g) & 3], t[(2 + g) & 3], t[(3 + g) & 3]);
            }
        }
    }
    // The rest of the lane's row: the tile's first elements; the unit that both warps
    // share; at the row's end, or the tile's, the last ones.
    if (row0 + lane < p.M) {
        uint16_t *to = first + static_cast<int64_t>(lane) * p.N + HALF * 64 - shift;
        const int past = HALF == 1 && left && shift > 0 ? 72 : shift + 64;  // this half's last element, and one
        const int end = shift + cols < past ? shift + cols : past;
        const int tail = end / 8 * 8;
        if (HALF == 0 && left && shift > 0) {
            const int even = shift + (shift & 1);
            if (end >= 8) {
                if (shift & 1) to[shift] = static_cast<uint16_t>(*place(shift / 2) >> 16);
                if (even & 2) *reinterpret_cast<uint32_t *>(to + even) = *place(even / 2);
                if (shift <= 4) *reinterpret_cast<uint2 *>(to + 4) = make_uint2(*place(2), *place(3));
            } else {
                for (int e = shift; e < end; ++e) to[e] = static_cast<uint16_t>(*place(e / 2) >> (e % 2 * 16));
            }
        }
        if (HALF == 1 && end == 72) {
            *reinterpret_cast<uint4 *>(to + 64) = make_uint4(*place(32), *place(33), *place(34), *place(35));
        } else if (cols > 0 && (HALF == 1 || (cols <= 64 && (tail > 0 || shift == 0)))) {
            // not where the next half continues the unit, nor the first unit (above, or the left warp's)
            uint16_t *d = to + tail;
            const int n = end - tail, word = tail / 2;
            if (n & 4) *reinterpret_cast<uint2 *>(d) = make_uint2(*place(word), *place(word + 1));
            if (n & 2) *reinterpret_cast<uint32_t *>(d + (n & 4)) = *place(word + (n & 4) / 2);
            if (n & 1) d[n & 6] = static_cast<uint16_t>(*place(word + (n & 6) / 2));
        }
    }
    __syncwarp();
}

template <bool NV>
__global__ void __launch_bounds__(Fp4Pair<NV>::THREADS, 1)
    fp4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                    const __grid_constant__ CUtensorMap tmD, const Fp4Params p) {
    using C = Fp4Pair<NV>;
    using S = typename C::S;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
    const int lane = static_cast<int>(threadIdx.x) % 32;
    const int rank = static_cast<int>(ptx::cluster_ctarank());
    const bool leader = rank == 0;
    const int cluster = static_cast<int>(blockIdx.x) / 2, clusters = static_cast<int>(gridDim.x) / 2;
    const int tiles = p.m_tiles * p.n_tiles;

    const uint32_t bar_full = base + C::OFF_BAR, bar_empty = bar_full + 8 * C::STAGES;
    const uint32_t bar_tfull = bar_empty + 8 * C::STAGES;  // [2] accumulator complete
    const uint32_t bar_share = bar_tfull + 16;             // shared columns read
    const uint32_t bar_drain = bar_share + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);

    if (warp == 0 && lane == 0) {
        ptx::prefetch_tensormap(&tmA);
        ptx::prefetch_tensormap(&tmB);
        ptx::prefetch_tensormap(&tmSA);
        ptx::prefetch_tensormap(&tmSB);
        ptx::prefetch_tensormap(&tmD);
        for (int s = 0; s < C::STAGES; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        ptx::mbar_init(bar_tfull, 1);
        ptx::mbar_init(bar_tfull + 8, 1);
        ptx::mbar_init(bar_share, 2 * C::EPI_WARPS);  // the epilogue warps of both CTAs
        ptx::mbar_init(bar_drain, 1);
        *abort_flag = 0;
        ptx::fence_mbarrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc<2>(ptx::smem_u32(tmem_slot), 512);
        ptx::tmem_relinquish<2>();
    }
    ptx::tcgen05_fence_before();
    ptx::cluster_sync();
    ptx::tcgen05_fence_after();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();

    auto tile_of = [&](int item) {
        return gemm_f16::work_of(item, p.m_tiles, p.n_tiles, p.raster_group, tiles, p.k_tiles, 1, 256);
    };
    if (warp == 0) {
        if (ptx::elect_one()) {
            ptx::griddep_wait();
            PipelineState ring(C::STAGES, (p.debug_flags & 1u) ? 0u : 1u);
            bool ok = true;
            uint32_t seq = 0;
            for (int item = cluster; ok && item < tiles; item += clusters, ++seq) {
                const WorkItem w = tile_of(item);
                const int32_t a_row = w.m_idx * 256 + rank * 128, b_row = w.n_idx * 256 + rank * 128;
                for (int kt = 0; kt < p.k_tiles; ++kt) {
                    if (!wait_bounded(bar_empty + 8 * ring.stage, ring.phase, abort_flag, p.timeout_ns,
                                      gemm_f16::kRoleProducer, seq)) {
                        ok = false;
                        break;
                    }
                    const int s = ring.stage;
                    const uint32_t full = bar_full + 8 * s, full_leader = ptx::mapa(full, 0);
                    if (leader) ptx::mbar_arrive_expect_tx(full, S::TX);
                    ptx::tma_load_2d_pair(base + C::OFF_A + s * S::A_BYTES, &tmA, full_leader, kt * 128, a_row);
                    ptx::tma_load_2d_pair(base + C::OFF_B + s * S::B_BYTES, &tmB, full_leader, kt * 128, b_row);
                    ptx4::tma_load_3d_pair(base + C::OFF_SFA + s * S::SFA_BYTES, &tmSA, full_leader, 0,
                                           kt * S::SF_TILES, w.m_idx * 2 + rank);
                    ptx4::tma_load_3d_pair(base + C::OFF_SFB + s * S::SFB_BYTES, &tmSB, full_leader, 0,
                                           kt * S::SF_TILES, w.n_idx * 2);
                    ring.advance();
                }
            }
            if (!ok) {
                const uint64_t t0 = ptx::globaltimer_ns();
                while (ptx::globaltimer_ns() - t0 < 20000) ptx::nanosleep(1000);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader && ptx::elect_one()) {
            PipelineState ring(C::STAGES, 0u);
            PipelineState share(1, 1u);  // the first tile waits for nothing
            bool ok = true;
            uint32_t seq = 0, stage_seq = 0;
            for (int item = cluster; ok && item < tiles; item += clusters, ++seq) {
                const uint32_t d = tmem_base + (seq % 2 ? C::ACC1 : 0);
                for (int kt = 0; kt < p.k_tiles; ++kt, ++stage_seq) {
                    if (!wait_bounded(bar_full + 8 * ring.stage, ring.phase, abort_flag, p.timeout_ns,
                                      gemm_f16::kRoleMma, seq)) {
                        ok = false;
                        break;
                    }
                    ptx::tcgen05_fence_after();
                    const int s = ring.stage;
                    const uint32_t tsf = tmem_base + C::SF_COL + stage_seq % C::SF_BUFS * S::SF_COLS;
                    S::copy_scales(base + C::OFF_SFA + s * S::SFA_BYTES, base + C::OFF_SFB + s * S::SFB_BYTES, tsf);
                    if (kt == 0) {
                        // the previous tile's epilogue has read the columns both accumulators share
                        if (!wait_bounded(bar_share, share.phase, abort_flag, p.timeout_ns, gemm_f16::kRoleMma, seq)) {
                            ok = false;
                            break;
                        }
                        share.advance();
                        ptx::tcgen05_fence_after();
                    }
                    S::multiply(base + C::OFF_A + s * S::A_BYTES, base + C::OFF_B + s * S::B_BYTES, tsf, d, kt == 0);
                    ptx::mma_commit<2>(bar_empty + 8 * s, 0x3);
                    ring.advance();
                }
                if (!ok) break;
                ptx::mma_commit<2>(bar_tfull + 8 * (seq % 2), 0x3);
            }
            ptx::mma_commit<2>(bar_drain, 0x1);
            wait_bounded(bar_drain, 0, abort_flag, p.timeout_ns, gemm_f16::kRoleMma, 0xFFFFFFFFu, false);
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3, half = (warp - 2) / 4;  // of the CTA's rows, of the tile's columns
        const uint32_t rows_base = base + C::OFF_D + static_cast<uint32_t>((warp - 2) * C::EPI_ROWS);
        const uint32_t stage_base = base + C::OFF_D + static_cast<uint32_t>((warp - 2) * C::EPI_BUF);
        const uint32_t share_leader = ptx::mapa(bar_share, 0);
        uint32_t seq = 0;
        for (int item = cluster; item < tiles; item += clusters, ++seq) {
            const WorkItem w = tile_of(item);
            const int32_t row0 = w.m_idx * 256 + rank * 128 + quarter * 32, col0 = w.n_idx * 256 + half * 128;
            bool ok = true;
            if (lane == 0) {
                ok = wait_bounded(bar_tfull + 8 * (seq % 2), seq / 2 % 2, abort_flag, p.timeout_ns,
                                  gemm_f16::kRoleEpilogue, seq);
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (!ok) break;
            if (seq == 0) ptx::griddep_wait();
            ptx::tcgen05_fence_after();
            const bool second = seq % 2;
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + (second ? C::ACC1 : 0) +
                                   static_cast<uint32_t>(half * 128);
            // 64-column chunks of this warp's half, the shared columns first: the last
            // ones of the first accumulator, the first ones of the second.  The half
            // without any hands over what it has read with the tile before.
            const bool shares = half == (second ? 0 : 1);
            auto chunk_at = [&](int i) { return second ? i : 1 - i; };
            auto hand_over = [&]() {
                ptx::tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) ptx4::mbar_arrive_cluster_relaxed(share_leader);
            };
            constexpr int kShared = (C::OVER + 63) / 64;  // chunks that hold shared columns
            static_assert(kShared <= 2, "in one half");
            if (!shares) hand_over();
            if (p.d_type != LINEAR_F32) {
                // the whole slice in registers, rounded, before any of it is stored
                uint32_t h[2][32];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t col = static_cast<uint32_t>(chunk_at(i) * 64);
                    uint32_t lo[32], hi[32];
                    ptx::tmem_ld_32x32b_x32(taddr + col, lo);
                    ptx::tmem_ld_32x32b_x32(taddr + col + 32, hi);
                    ptx::tmem_wait_ld();
                    if (shares && i == kShared - 1) hand_over();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        h[i][j] = scaled16(p, lo[2 * j], lo[2 * j + 1]);
                        h[i][16 + j] = scaled16(p, hi[2 * j], hi[2 * j + 1]);
                    }
                }
                if (!p.tma_store) {
                    uint32_t after[4] = {};
                    if (half == 0) {
                        uint32_t v[16];
                        ptx::tmem_ld_32x32b_x16(taddr + 128, v);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 4; ++j) after[j] = scaled16(p, v[2 * j], v[2 * j + 1]);
                    }
                    uint8_t *rows = smem + (rows_base - base);
                    uint32_t w[32];  // the low 64 columns, then the high ones
#pragma unroll
                    for (int j = 0; j < 32; ++j) w[j] = second ? h[0][j] : h[1][j];
                    store_unaligned<0, C::ROW_PITCH>(p, rows, w, 0u, after, half == 0, lane, row0, col0);
                    const uint32_t before = w[31];
#pragma unroll
                    for (int j = 0; j < 32; ++j) w[j] = second ? h[1][j] : h[0][j];
                    store_unaligned<1, C::ROW_PITCH>(p, rows, w, before, after, half == 0, lane, row0, col0);
                    continue;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int32_t col = col0 + chunk_at(i) * 64;
                    if (lane == 0) ptx::bulk_wait_group_read<0>();
                    __syncwarp();
                    const uint32_t row_addr = stage_base + static_cast<uint32_t>(lane) * 128u;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t unit = static_cast<uint32_t>(j) ^ (static_cast<uint32_t>(lane) & 7u);
                        ptx::st_shared_v4(row_addr + unit * 16u, h[i][4 * j], h[i][4 * j + 1], h[i][4 * j + 2],
                                          h[i][4 * j + 3]);
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (row0 < p.M && col < p.N) ptx::tma_store_2d(&tmD, stage_base, col, row0);
                        ptx::bulk_commit_group();
                    }
                }
            } else {
                // fp32: 32 columns at a time through 32 x 32 floats of staging (row r's
                // column c at c ^ r), read back by rows, one element a lane
                float *stage = reinterpret_cast<float *>(smem + (stage_base - base));
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    const int c32 = second ? i : 3 - i;
                    uint32_t v[32];
                    ptx::tmem_ld_32x32b_x32(taddr + c32 * 32, v);
                    ptx::tmem_wait_ld();
                    if (shares && i == 2 * kShared - 1) hand_over();
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float2 d = scaled(p, v[j], v[j + 1]);
                        stage[lane * 32 + (j ^ lane)] = d.x;
                        stage[lane * 32 + ((j + 1) ^ lane)] = d.y;
                    }
                    __syncwarp();
                    const int32_t col = col0 + c32 * 32 + lane;
                    if (col < p.N) {
#pragma unroll 4
                        for (int r = 0; r < 32; ++r) {
                            if (row0 + r < p.M) {
                                store_d(p.D, p.d_type, static_cast<int64_t>(row0 + r) * p.N + col,
                                        stage[r * 32 + (lane ^ r)]);
                            }
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (lane == 0) ptx::bulk_wait_group_read<0>();
        __syncwarp();
    }
    // the pair's CTAs done with TMEM and with each other's barriers (nothing in memory
    // is published here, so the arrival waits for no store)
    ptx::tcgen05_fence_before();
    ptx::cluster_arrive_relaxed();
    ptx::cluster_wait();
    if (warp == 1) {
        ptx::tcgen05_fence_after();
        ptx::tmem_dealloc<2>(tmem_base, 512);
    }
}

}  // namespace linear_ops
