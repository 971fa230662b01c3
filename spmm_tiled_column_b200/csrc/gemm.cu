// gemm.cu -- prefill products with an epilogue, the gated block, and the gradients, as dense
// products on tcgen05 SM pairs over the expanded weight:
//   spw_spmm_ep            Y = act(X W^T + bias) + residual
//   spw_spmm_ffn           H = act(X Wg^T) * (X Wu^T)
//   spw_spmm_ffn_backward  dX = dG Wg + dU Wu, and dG^T X, dU^T X at the kept positions
//   spw_spmm_backward      dX = dY W, and dY^T X at the kept positions
//
// For few tokens these calls take the direct form of spmm_direct.cu instead (choose_direct); the
// gradients of kept weights are computed here alone.
//
// Why expanded: spmm.cu decodes each weight tile into shared memory once per token tile, and
// the decode, the operand's stores and the MMA's reads then share one SM's shared-memory
// bandwidth.  Here expand_kernel writes the dense weight once into the workspace (a
// write of 2 N K bytes, most of it still in L2 when it is read), and the product runs as a
// plain dense GEMM whose operands come by TMA alone; a gradient needs the weight along its
// other dimension, which the same expanded copy serves as an MN-major operand.  Bound by the
// tensor cores: 4096 x 4096 at 4096 tokens 101 us (1360 TFLOP/s; a dense library product 95),
// 4096 x 11008 at 2048 tokens 138 us (121), and 12 and 27 us for their expansion.
//
// The product: a cluster of two CTAs (an SM pair) computes a 256 x BN tile (BN = 256 or 128)
// with tcgen05.mma.cta_group::2: each CTA holds 128 rows of A, half of B and 128 rows of the
// fp32 accumulator in its own tensor memory (two accumulators of BN columns, so that the
// epilogue of one tile runs under the MMAs of the next).  Persistent: pair p takes the units
// p, p + pairs, ...; a unit is an output tile, or one of `parts` pieces of its reduction when
// there are too few tiles; pieces go to fp32 partials in the workspace and the last CTA of a
// tile to arrive adds them in order (deterministic) and runs the epilogue.
//   warp 0, lane 0: TMA loads of this CTA's operand halves, `stages` deep; both CTAs' loads
//     of a stage count on one barrier of rank 0 (a relay through rank 1, with an arrive at
//     cluster scope for each stage, cost 0.3 us a step).
//   warp 1: rank 0 issues the MMAs of the pair and commits each stage back to both CTAs.
//   warps 2..9: epilogue; warp w reads the TMEM lanes 32 (w % 4).., one half of the columns.
// Every wait is bounded and polls the pair's abort flags, as in spmm.cu.
#include <string.h>

#include <mutex>

#include "spw_prefill.cuh"
#include "spw_tcgen05.cuh"

namespace spw {
namespace {

// ------------------------------------------------------------------ expansion
// 32 bytes to a 32-byte aligned address.
__device__ inline void st_global_32b(void* at, const uint32_t (&a)[4], const uint32_t (&b)[4]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(a[0]), "r"(a[1]), "r"(a[2]),
                 "r"(a[3]), "r"(b[0]), "r"(b[1]), "r"(b[2]), "r"(b[3])
                 : "memory");
}

constexpr int kExpandWarps = 8;
// A warp's records {bits, end of the half's values} of 64 columns: low halves, high halves (16
// bytes off, in other banks).
constexpr uint32_t kRecHalf = 64 * 8 + 16;
constexpr uint32_t kRecBytes = 2 * kRecHalf;

struct ExpandLayer {
    const uint64_t* bitmaps;
    const uint32_t* tileptr;
    const uint16_t* values;
    uint64_t values_units;
    uint32_t max_units;
    uint16_t* out;
    int n_ktiles;
    long long n_tiles;
};

struct ExpandParams {
    ExpandLayer L[2];
    long long tiles;    // both layers
    int strips, ktp;    // strips of an output block; blocks of a row of blocks
    uint32_t warp_smem;
    int* status;
    uint32_t* clear;    // counters of the products that follow, cleared here
    uint32_t n_clear;
};

// One warp writes one 64 x 64 tile of the dense weight, in the blocks that the product reads: p.strips
// strips by one k-tile, [8 columns][row][8 columns of it], 16 bytes a row.  Lane l has the rows 2l and
// 2l+1, so a store of the warp covers 1024 bytes.  Bound by memory: the compressed weight in, 2 bytes an
// entry out (4096 x 8192 at 50 %: 105 MB in 20 us, 5.2 TB/s).
__global__ void __launch_bounds__(32 * kExpandWarps) expand_kernel(const __grid_constant__ ExpandParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    pdl_launch_dependents();  // the product may set itself up; it waits for this grid's end
    for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < p.n_clear; i += gridDim.x * blockDim.x) p.clear[i] = 0u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned char* mine = smem + (size_t)warp * p.warp_smem;
    unsigned char* rec = mine;
    const int up = 30 - 2 * (lane & 15);
    const uint32_t above = 0xFFFFFFFEu << (2 * (lane & 15));
    const uint4* recp = (const uint4*)(rec + (lane < 16 ? 0u : kRecHalf));
    unsigned char* vals = mine + kRecBytes;  // 16 bytes of slack first: see the loads below
    const uint32_t vals_s = smem_u32(vals) + 16u;
    for (long long i = (long long)blockIdx.x * kExpandWarps + warp; i < p.tiles;
         i += (long long)gridDim.x * kExpandWarps) {
        const ExpandLayer& L = p.L[i >= p.L[0].n_tiles ? 1 : 0];
        const long long t = i >= p.L[0].n_tiles ? i - p.L[0].n_tiles : i;
        const uint32_t u0 = __ldg(L.tileptr + t), u1 = __ldg(L.tileptr + t + 1);
        const uint4 bw = __ldg((const uint4*)(L.bitmaps + t * kTileCols) + lane);  // columns 2l, 2l+1
        const int cl0 = __popc(bw.x), c0 = cl0 + __popc(bw.y);
        const int cl1 = __popc(bw.z), c1 = cl1 + __popc(bw.w);
        const int incl = warp_inclusive_scan(c0 + c1, lane);
        const int total = __shfl_sync(0xffffffffu, incl, 31);
        // the tile's values fill u1 - u0 units of 8: anything else than its bitmaps' count
        // rounded up, or a range outside the section, is reported and decoded as empty
        bool ok = u1 >= u0 && u1 <= L.values_units && u1 - u0 <= L.max_units &&
                  (uint32_t)(total + 7) / 8u == u1 - u0;
        if (!ok && lane == 0) raise_status(p.status, SPW_ERR_FORMAT);
        __syncwarp();
        if (ok) {
            const uint4* src = (const uint4*)(L.values + (size_t)u0 * 8);
            for (uint32_t j = lane; j < u1 - u0; j += 32) ((uint4*)(vals + 16))[j] = __ldg(src + j);
            const uint32_t a0 = vals_s + 2u * (uint32_t)(incl - c0 - c1), a1 = a0 + 2u * (uint32_t)c0;
            *(uint4*)(rec + 16 * lane) = make_uint4(bw.x, a0 + 2u * (uint32_t)cl0, bw.z, a1 + 2u * (uint32_t)cl1);
            *(uint4*)(rec + kRecHalf + 16 * lane) = make_uint4(bw.y, a1, bw.w, a1 + 2u * (uint32_t)c1);
        }
        __syncwarp();
        const long long strip = t / L.n_ktiles;
        const int kt = (int)(t - strip * L.n_ktiles);
        unsigned char* out = (unsigned char*)L.out + ((strip / p.strips) * p.ktp + kt) * (size_t)(p.strips * 8192) +
                             (strip % p.strips) * 1024 + 32 * lane;
#pragma unroll
        for (int g = 0; g < 8; g++) {
            uint32_t o0[4] = {0u, 0u, 0u, 0u}, o1[4] = {0u, 0u, 0u, 0u};
            if (ok) {
#pragma unroll
                for (int c = 0; c < 4; c++) decode_pair(recp[4 * g + c], above, up, o0[c], o1[c]);
            }
            st_global_32b(out + (size_t)g * (p.strips * 1024), o0, o1);
        }
        __syncwarp();
    }
}

// ------------------------------------------------------------------ the product
constexpr int kCtaRows = 128;  // accumulator rows per CTA; 256 per pair
constexpr int kBK = 64;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kStageBlocks = 2;  // blocks of 64 along the reduction in a stage
constexpr int kMaxStages = 8;
constexpr uint32_t kABytes = kCtaRows * kBK * 2;  // 16 KB
constexpr int kAccCols = 256;                     // columns between the two accumulators
constexpr int kSmemLimit = 227 * 1024;

struct GemmParams {
    int m_tiles, n_tiles, group_m, problem_tiles;
    int n_units, parts;
    int ksteps, kseg;  // reduction blocks of 64 of a tile; those of its first segment (kDx)
    int BN, stages;
    uint32_t block_bytes, stage_bytes, off_bar;  // this CTA's operands, 64 deep; kStageBlocks of them
    uint32_t off_stage;  // the epilogue warps' blocks
    long long wait_limit;
    int* status;
    uint32_t* counters;  // arrivals per split tile and rank
    float* partials;     // [split tile][part][rank][BN][128]
    PrefillOut o;
    // kDv: per weight, its pattern and the packed gradient
    const uint64_t* bitmaps[2];
    const uint32_t* tileptr[2];
    uint64_t values_units[2];
    uint16_t* dv[2];
    int n_strips, n_ktiles;
    int ktp;             // expanded weight: blocks in a row of blocks
};

struct Unit {
    int prob, mt, nt, k0, k1;
    int stile, part;  // of a split tile; stile < 0: whole
};

// Tiles run m fastest inside bands of group_m row tiles, so that the pairs at work at one
// time share a few column tiles' operands in L2.
__device__ inline Unit unit_of(const GemmParams& p, int u) {
    Unit w;
    int tile = u;
    w.stile = -1;
    w.part = 0;
    w.k0 = 0;
    w.k1 = p.ksteps;
    if (p.parts > 1) {
        tile = w.stile = u / p.parts;
        w.part = u - tile * p.parts;
        w.k0 = (int)((long long)w.part * p.ksteps / p.parts);
        w.k1 = (int)((long long)(w.part + 1) * p.ksteps / p.parts);
    }
    w.prob = tile / p.problem_tiles;
    const int t = tile - w.prob * p.problem_tiles;
    const int band = t / (p.group_m * p.n_tiles);
    const int first = band * p.group_m;
    const int gm = min(p.group_m, p.m_tiles - first);
    const int r = t - band * p.group_m * p.n_tiles;
    w.nt = r / gm;
    w.mt = first + (r - w.nt * gm);
    return w;
}

// Blocks of 64 along the reduction that the stage starting at block k holds: fewer at the end
// of the unit's range or (kDx) of a segment.
template <int MODE>
__device__ inline int blocks_at(const GemmParams& p, int k, int k1) {
    int n = min(kStageBlocks, k1 - k);
    if (MODE == kDx && k < p.kseg) n = min(n, p.kseg - k);
    return n;
}

// The same barrier in both CTAs of the pair, once the MMAs issued so far have completed.
__device__ inline void umma_commit_pair_multicast(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// MN-major operand, 128-byte swizzle: blocks of 64 (M or N) x 64 (K), each K row 128 bytes;
// 8-row groups along K 1024 bytes apart, the 64-wide blocks 8192 bytes apart.
__device__ inline uint64_t umma_desc_mn_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFF);
    d |= (uint64_t)(8192 >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// This CTA's load, counted on a barrier of the pair that may be the other CTA's (no multicast).
__device__ inline void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"((uint64_t)map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// Counts bytes on a barrier without a copy.
__device__ inline void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Joins the epilogue warps (named barrier 1) and tells whether all of them hold `ok`.
__device__ inline bool epi_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.and.pred p, 1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(ok ? 1u : 0u), "n"(32 * kEpiWarps)
        : "memory");
    return r != 0;
}

__device__ inline uint32_t pack2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *(const uint32_t*)&h;
}

// Adds 32 values of a bias to columns col .. col+31.
__device__ inline void add_bias(const uint16_t* bias, int col, int cols, float (&v)[32]) {
    if (col + 32 <= cols) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint4 r = *(const uint4*)(bias + col + 8 * j);
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float2 f = __half22float2(*(const __half2*)&w[e]);
                v[8 * j + 2 * e] += f.x;
                v[8 * j + 2 * e + 1] += f.y;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; j++)
            if (col + j < cols) v[j] += __half2float(__ushort_as_half(bias[col + j]));
    }
}

// Writes a warp's 32 x 32 block (lane l holds row l, columns col .. col+31) to rows row0 .. of
// a row-major fp16 matrix, plus the residual's block if there is one.  Where 16-byte accesses
// are allowed each lane writes its own row.  Elsewhere the block goes through the warp's piece
// of shared memory (rows 33 floats apart: no two lanes in one bank), so that a row's 64 bytes
// go out together: with a lane writing 2 bytes at a time of its own row, a ragged leading
// dimension took longer than the whole product (500 x 1300, 4096 tokens: 34 us against 18; the
// aligned 4096 x 1024 takes 47 us through shared memory, 40 us without).
// pairs: even leading dimensions, so two columns a lane.
__device__ inline void store_block(float* stage, int lane, uint16_t* Y, int ldy, const uint16_t* residual, int ldr, int row0,
                                   int rows, int col, int cols, bool vec, bool pairs, const float (&v)[32]) {
    if (vec && col + 32 <= cols) {
        if (row0 + lane >= rows) return;
        const size_t r = (size_t)(row0 + lane);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            uint4 q = make_uint4(0u, 0u, 0u, 0u);
            if (residual) q = *(const uint4*)(residual + r * ldr + col + 8 * j);
            const uint32_t in[4] = {q.x, q.y, q.z, q.w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                float2 f = make_float2(v[8 * j + 2 * e], v[8 * j + 2 * e + 1]);
                if (residual) {
                    const float2 a = __half22float2(*(const __half2*)&in[e]);
                    f.x += a.x;
                    f.y += a.y;
                }
                o[e] = pack2(f.x, f.y);
            }
            *(uint4*)(Y + r * ldy + col + 8 * j) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        return;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 32; j++) stage[lane * 33 + j] = v[j];
    __syncwarp();
    const int n = min(32, rows - row0);
    if (pairs) {
        const int c = 2 * (lane & 15), hi = lane >> 4;
        if (col + c + 1 < cols) {
#pragma unroll 8
            for (int i = hi; i < n; i += 2) {
                const size_t r = (size_t)(row0 + i);
                float2 f = make_float2(stage[i * 33 + c], stage[i * 33 + c + 1]);
                if (residual) {
                    const float2 q = __half22float2(*(const __half2*)(residual + r * ldr + col + c));
                    f.x += q.x;
                    f.y += q.y;
                }
                *(uint32_t*)(Y + r * ldy + col + c) = pack2(f.x, f.y);
            }
        } else if (col + c < cols) {
            for (int i = hi; i < n; i += 2) {
                const size_t r = (size_t)(row0 + i);
                float f = stage[i * 33 + c];
                if (residual) f += __half2float(__ushort_as_half(residual[r * ldr + col + c]));
                Y[r * ldy + col + c] = __half_as_ushort(__float2half_rn(f));
            }
        }
    } else if (col + lane < cols) {
#pragma unroll 8
        for (int i = 0; i < n; i++) {
            const size_t r = (size_t)(row0 + i);
            float f = stage[i * 33 + lane];
            if (residual) f += __half2float(__ushort_as_half(residual[r * ldr + col + lane]));
            Y[r * ldy + col + lane] = __half_as_ushort(__float2half_rn(f));
        }
    }
}

// A tile whose bitmaps and pointers disagree counts as empty: zeros over what it claims, or, where
// that is no tile's size or leaves the section, over its bitmaps' number of units behind its start
// and before its end (one of the two pointers may be right).
__device__ __noinline__ void zero_disagreeing(uint16_t* dv, uint64_t section, uint32_t u0, uint32_t u1, uint32_t n, int lane) {
    auto zero = [&](uint64_t first, uint64_t count) {
        if (first + count > section) return;
        for (uint64_t i = lane; i < count; i += 32) ((uint4*)dv)[first + i] = make_uint4(0u, 0u, 0u, 0u);
    };
    if (u1 >= u0 && u1 <= section && u1 - u0 <= kStripRows * kTileCols / 8) {
        zero(u0, u1 - u0);
    } else {
        zero(u0, n);
        if (u1 >= n) zero(u1 - n, n);
    }
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap ta0, const __grid_constant__ CUtensorMap ta1,
            const __grid_constant__ CUtensorMap tb0, const __grid_constant__ CUtensorMap tb1,
            const __grid_constant__ GemmParams p) {
    constexpr bool A_MN = MODE == kDv;                  // A's rows lie along its memory rows
    constexpr bool B_MN = MODE == kDx || MODE == kDv;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
    const int S = p.stages;

    uint64_t* full = (uint64_t*)(smem + p.off_bar);  // on rank 0: both CTAs' loads of a stage
    uint64_t* empty = full + kMaxStages;
    uint64_t* acc_full = empty + kMaxStages;
    uint64_t* acc_empty = acc_full + 2;         // on rank 0: both CTAs' epilogue warps
    uint64_t* drain = acc_empty + 2;
    uint32_t* tmem_slot = (uint32_t*)(drain + 1);
    volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
    volatile uint32_t* last_flag = (volatile uint32_t*)(tmem_slot + 2);
    volatile uint32_t* peer_issued = (volatile uint32_t*)(tmem_slot + 3);  // see the drain

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; i++) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_u32(&acc_full[i]), 1);
            mbar_init(smem_u32(&acc_empty[i]), 2 * kEpiWarps);
        }
        mbar_init(smem_u32(drain), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(2u * kAccCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t peer_abort = map_to_rank(smem_u32((const void*)abort_flag), rank ^ 1u);
    auto abort_both = [&]() {
        flag_abort(abort_flag, p.status);
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_abort), "r"(1) : "memory");
    };
    const int half_cols = p.BN / 2;

    // Launched while the kernel before it in the same call still runs.  kEp, kFfn, kDx read what
    // that kernel writes (the expansion; dG and dU stand before it): the producer waits for
    // its end, then lets the next kernel of the call start.  kDv reads nothing of the kernel
    // before it (the input's gradient), which waited itself for dG and dU before it let kDv
    // start; it only must not end before it, see below.
    uint32_t issued = 0;  // producer: stages loaded
    if (MODE != kDv && threadIdx.x == 0) {
        pdl_wait();
        pdl_launch_dependents();
    }
    if (warp == 0) {
        if (lane == 0) {
            const uint32_t full0 = map_to_rank(smem_u32(&full[0]), 0u);
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int u = pair; u < p.n_units && ok; u += pairs) {
                const Unit w = unit_of(p, u);
                const int arow = w.mt * 2 * kCtaRows + kCtaRows * (int)rank;
                const int brow = MODE == kFfn ? w.nt * half_cols : w.nt * p.BN + half_cols * (int)rank;
                for (int k = w.k0, n; k < w.k1; k += n) {
                    n = blocks_at<MODE>(p, k, w.k1);
                    if (issued >= S && !wait_or_abort(smem_u32(&empty[s]), ph ^ 1u, abort_flag, p.wait_limit)) {
                        abort_both();
                        ok = false;
                        break;
                    }
                    const uint32_t bar = full0 + 8u * (uint32_t)s;
                    // the other CTA's bytes may land before this; the phase waits for the arrival
                    if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full[s]), 2u * (uint32_t)n * p.block_bytes);
                    const bool second = MODE == kDx ? k >= p.kseg : w.prob != 0;
                    const CUtensorMap* ma = second ? &ta1 : &ta0;
                    const CUtensorMap* mb = (MODE == kFfn ? rank != 0 : MODE == kDx && second) ? &tb1 : &tb0;
                    for (int i = 0; i < n; i++) {
                        const uint32_t a = sbase + (uint32_t)s * p.stage_bytes + (uint32_t)i * kABytes;
                        const uint32_t b = sbase + (uint32_t)s * p.stage_bytes + kStageBlocks * kABytes + (uint32_t)(i * half_cols * 128);
                        const int kc = kBK * (MODE == kDx && second ? k + i - p.kseg : k + i);
                        if constexpr (A_MN) {
                            tma_load_2d_pair(a, ma, arow, kc, bar);
                            tma_load_2d_pair(a + 8192u, ma, arow + 64, kc, bar);
                        } else {
                            tma_load_2d_pair(a, ma, kc, arow, bar);
                        }
                        if constexpr (MODE == kDv) {
                            for (int j = 0; j < half_cols / 64; j++)
                                tma_load_2d_pair(b + 8192u * j, mb, brow + 64 * j, kc, bar);
                        } else if constexpr (MODE == kDx) {
                            tma_load_2d_pair(b, mb, 0, 64 * (kc / kBK * p.ktp) + brow, bar);
                        } else {
                            tma_load_2d_pair(b, mb, 0, (brow / half_cols * p.ktp + k + i) * half_cols, bar);
                        }
                    }
                    issued++;
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        // ------------------------------------------------------------ MMAs
        const uint32_t idesc = idesc_f16(2 * kCtaRows, p.BN) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
        const uint32_t b0 = sbase + kStageBlocks * kABytes;
        const uint64_t ad0 = A_MN ? umma_desc_mn_sw128(sbase) : umma_desc_sw128(sbase);
        const uint64_t bd0 = MODE == kDv   ? umma_desc_mn_sw128(b0)
                             : MODE == kDx ? umma_desc_plain(b0, 128, 1024)
                                           : umma_desc_plain(b0, 16u * half_cols, 128);
        // from a slice of 16 along the reduction to the next
        const uint32_t da = A_MN ? 2048u : 32u, db = MODE == kDv ? 2048u : MODE == kDx ? 256u : 32u * half_cols;
        int s = 0, it = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int u = pair; u < p.n_units && ok; u += pairs, it++) {
            const Unit w = unit_of(p, u);
            const int a = it & 1;
            if (it >= 2) {
                ok = __all_sync(0xffffffffu, wait_or_abort_cluster(smem_u32(&acc_empty[a]), (uint32_t)(((it >> 1) & 1) ^ 1),
                                                                   abort_flag, p.wait_limit));
                if (!ok) {
                    if (lane == 0) abort_both();
                    break;
                }
            }
            tc_fence_after();
            for (int k = w.k0, n; k < w.k1; k += n) {
                n = blocks_at<MODE>(p, k, w.k1);
                ok = __all_sync(0xffffffffu, wait_or_abort(smem_u32(&full[s]), ph, abort_flag, p.wait_limit));
                if (!ok) {
                    if (lane == 0) abort_both();
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t so = (uint32_t)s * p.stage_bytes;
                    for (int i = 0; i < n; i++) {
#pragma unroll
                        for (int j = 0; j < kBK / 16; j++)
                            umma_f16_pair(tmem + (uint32_t)(kAccCols * a), ad0 + ((so + (uint32_t)i * kABytes + da * j) >> 4),
                                          bd0 + ((so + (uint32_t)(i * half_cols * 128) + db * j) >> 4), idesc,
                                          (k > w.k0 || i > 0 || j > 0) ? 1u : 0u);
                    }
                    umma_commit_pair_multicast(smem_u32(&empty[s]));
                    if (k + n >= w.k1) umma_commit_pair_multicast(smem_u32(&acc_full[a]));
                }
                __syncwarp();
                if (++s == S) { s = 0; ph ^= 1u; }
            }
        }
        if (elect_one()) umma_commit_pair_local(smem_u32(drain));
        __syncwarp();
        (void)mbar_drain(smem_u32(drain), 0);  // every issued MMA has completed
        __syncwarp();
    } else if (warp >= 2) {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3, side = (warp - 2) >> 2;
        const int row = 32 * quarter + lane;  // accumulator row of this CTA
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const uint32_t empty0 = map_to_rank(smem_u32(&acc_empty[0]), 0u);
        int it = 0;
        for (int u = pair; u < p.n_units; u += pairs, it++) {
            const Unit w = unit_of(p, u);
            const int a = it & 1;
            bool ok = __all_sync(0xffffffffu, wait_or_abort(smem_u32(&acc_full[a]), (uint32_t)((it >> 1) & 1),
                                                            abort_flag, p.wait_limit));
            if (!ok && lane == 0) abort_both();
            if (!epi_all(ok)) break;  // all warps or none: the barriers below need every one
            tc_fence_after();
            const uint32_t acc = tmem + lanes + (uint32_t)(kAccCols * a);
            const float* part = nullptr;
            if (w.stile >= 0) {
                // A piece of the reduction: publish it; the last piece of the tile (of this
                // CTA's rows) goes on with the sum of all, the others are done.
                float* tile_part = p.partials + (((size_t)w.stile * p.parts) * 2 + rank) * (size_t)p.BN * kCtaRows;
                float* out = tile_part + (size_t)w.part * 2 * p.BN * kCtaRows;
                const bool rows_in = w.mt * 2 * kCtaRows + kCtaRows * (int)rank + 32 * quarter < p.o.rows;
                for (int c = side * half_cols; c < (side + 1) * half_cols && rows_in; c += 32) {
                    uint32_t r[32];
                    tmem_ld32(acc + (uint32_t)c, r);
#pragma unroll
                    for (int j = 0; j < 32; j++) out[(size_t)(c + j) * kCtaRows + row] = __uint_as_float(r[j]);
                }
                tc_fence_before();
                __threadfence();
                (void)epi_all(true);  // every warp's partials before warp 2's arrival
                if (lane == 0) mbar_arrive_cluster(empty0 + 8u * a);
                if (warp == 2 && lane == 0) {
                    uint32_t* c = p.counters + 2 * w.stile + rank;
                    *last_flag = atom_add_acq_rel_gpu(c, 1u) == (uint32_t)(p.parts - 1) ? 1u : 0u;
                }
                (void)epi_all(true);
                const bool last = *last_flag != 0;
                (void)epi_all(true);  // read by all before the next unit writes it
                if (!last) continue;
                __threadfence();
                part = tile_part;
            }
            // 32 columns of this lane's row, from tensor memory or the sum of the pieces
            auto load = [&](int c, float (&v)[32]) {
                __syncwarp();
                if (!part) {
                    uint32_t r[32];
                    tmem_ld32(acc + (uint32_t)c, r);
#pragma unroll
                    for (int j = 0; j < 32; j++) v[j] = __uint_as_float(r[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; j++) v[j] = 0.0f;
                    for (int z = 0; z < p.parts; z++) {
                        const float* q = part + (size_t)z * 2 * p.BN * kCtaRows + (size_t)c * kCtaRows + row;
#pragma unroll
                        for (int j = 0; j < 32; j++) v[j] += __ldcg(q + (size_t)j * kCtaRows);
                    }
                }
            };
            const int r = w.mt * 2 * kCtaRows + kCtaRows * (int)rank + row;  // result row
            const bool rows_in = r - lane < p.o.rows;                        // some row of the warp's
            const int r0 = r - lane;  // the warp's first row
            float* stage = (float*)(smem + p.off_stage) + (warp - 2) * (32 * 33);
            if constexpr (MODE == kEp || MODE == kDx) {
                for (int c = side * half_cols; c < (side + 1) * half_cols && rows_in; c += 32) {
                    const int col = w.nt * p.BN + c;
                    if (col >= p.o.cols) break;
                    float v[32];
                    load(c, v);
                    if constexpr (MODE == kEp) {
                        if (p.o.bias) add_bias(p.o.bias, col, p.o.cols, v);
                        act_all(v, p.o.act);
                    }
                    store_block(stage, lane, p.o.Y, p.o.ldy, MODE == kEp ? p.o.residual : nullptr, p.o.ldr, r0, p.o.rows, col,
                                p.o.cols, (p.o.vec & 3) == 3, p.o.vec & 16, v);
                }
            } else if constexpr (MODE == kFfn) {
                // columns 0 .. BN/2-1 hold the gate, the others the up product of the same
                // BN/2 result columns
                for (int c = side * (half_cols / 2); c < (side + 1) * (half_cols / 2) && rows_in; c += 32) {
                    const int col = w.nt * half_cols + c;
                    if (col >= p.o.cols) break;
                    float g[32], v[32];
                    load(c, g);
                    load(half_cols + c, v);
                    if (p.o.G) {
                        store_block(stage, lane, p.o.G, p.o.ldg, nullptr, 0, r0, p.o.rows, col, p.o.cols, p.o.vec & 4, p.o.vec & 32, g);
                        store_block(stage, lane, p.o.U, p.o.ldu, nullptr, 0, r0, p.o.rows, col, p.o.cols, p.o.vec & 8, p.o.vec & 64, v);
                    }
                    act_all(g, p.o.act);
#pragma unroll
                    for (int j = 0; j < 32; j++) v[j] *= g[j];
                    store_block(stage, lane, p.o.Y, p.o.ldy, nullptr, 0, r0, p.o.rows, col, p.o.cols, p.o.vec & 1, p.o.vec & 16, v);
                }
            } else {
                // Packed gradient: row r of the weight is bit r % 64 of its strip's words; a
                // kept entry of column k stands after the kept entries of the tile's columns
                // before k and of the column's rows above it.
                const int strip = r / kStripRows;  // two quarters, one strip: warp-uniform
                const int hi = quarter & 1;        // this warp's half of the strip's rows
                for (int c = side * half_cols; c < (side + 1) * half_cols && rows_in; c += 64) {
                    float v[32];
                    const int kt = (w.nt * p.BN + c) / kTileCols;
                    const bool in = strip < p.n_strips && kt < p.n_ktiles;  // warp-uniform
                    uint32_t lo0 = 0, lo1 = 0, hi0 = 0, hi1 = 0, u0 = 0, u1 = 0;
                    int s0 = 0, s1 = 0, total = 0;
                    bool fits = false;
                    if (in) {
                        const size_t t = (size_t)strip * p.n_ktiles + kt;
                        u0 = __ldg(p.tileptr[w.prob] + t);
                        u1 = __ldg(p.tileptr[w.prob] + t + 1);
                        const uint4 bw = __ldg((const uint4*)(p.bitmaps[w.prob] + t * kTileCols) + lane);
                        lo0 = bw.x; hi0 = bw.y; lo1 = bw.z; hi1 = bw.w;  // columns 2l, 2l+1
                        const int c0 = __popc(lo0) + __popc(hi0), c1 = __popc(lo1) + __popc(hi1);
                        const int incl = warp_inclusive_scan(c0 + c1, lane);
                        total = __shfl_sync(0xffffffffu, incl, 31);
                        s0 = incl - c0 - c1;
                        s1 = s0 + c0;
                        fits = u1 >= u0 && u1 <= p.values_units[w.prob] && (uint32_t)(total + 7) / 8u == u1 - u0;
                        if (!fits) {
                            if (lane == 0) raise_status(p.status, SPW_ERR_FORMAT);
                            if (!hi) zero_disagreeing(p.dv[w.prob], p.values_units[w.prob], u0, u1, (uint32_t)(total + 7) / 8u, lane);
                        }
                    }
                    uint16_t* out = p.dv[w.prob] + (size_t)u0 * 8;
                    // the warp's words and the place of its first kept row in each column
                    const uint32_t w0 = hi ? hi0 : lo0, w1 = hi ? hi1 : lo1;
                    const int b0 = s0 + (hi ? __popc(lo0) : 0), b1 = s1 + (hi ? __popc(lo1) : 0);
                    const uint32_t below = lanemask_lt();
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        load(c + 32 * h, v);
#pragma unroll
                        for (int j = 0; j < 32; j++) {
                            const int src = 16 * h + (j >> 1);
                            const uint32_t bits = __shfl_sync(0xffffffffu, (j & 1) ? w1 : w0, src);
                            const int base = __shfl_sync(0xffffffffu, (j & 1) ? b1 : b0, src);
                            if (fits && ((bits >> lane) & 1u))
                                out[base + __popc(bits & below)] = __half_as_ushort(__float2half_rn(v[j]));
                        }
                    }
                    if (fits && !hi && lane < ((8 - (total & 7)) & 7)) out[total + lane] = 0;  // the filling
                }
            }
            if (!part) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(empty0 + 8u * a);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    // Rank 0's MMAs read both CTAs' shared memory, and each CTA arrives on the other's
    // barriers: neither leaves before both are here, with their copies landed.  On an abort the
    // producers may have stopped at different stages; rank 0, which owns the barriers, makes
    // up for the difference and waits for every stage that either has loaded.
    if (warp == 0 && lane == 0)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_rank(smem_u32((const void*)&peer_issued[rank]), 0u)),
                     "r"(issued)
                     : "memory");
    __syncthreads();
    cluster_sync_all();
    if (rank == 0 && warp == 0 && lane == 0 && *abort_flag) {
        const uint32_t mine = peer_issued[0], theirs = peer_issued[1];
        // (a stage's bytes follow from its place in the sequence of units)
        const uint32_t most = mine > theirs ? mine : theirs;
        uint32_t i = 0;
        for (int u = pair; u < p.n_units && i < most; u += pairs) {
            const Unit w = unit_of(p, u);
            for (int k = w.k0, n; k < w.k1 && i < most; k += n, i++) {
                n = blocks_at<MODE>(p, k, w.k1);
                if (i >= theirs)  // armed for both, loaded by this CTA alone
                    mbar_complete_tx(smem_u32(&full[i % S]), (uint32_t)n * p.block_bytes);
                else if (i >= mine)  // loaded by the other alone
                    mbar_arrive_expect_tx(smem_u32(&full[i % S]), (uint32_t)n * p.block_bytes);
            }
        }
        for (i = most > (uint32_t)S ? most - S : 0u; i < most; i++)
            (void)mbar_drain(smem_u32(&full[i % S]), (i / S) & 1u);
    }
    __syncwarp();
    __syncthreads();
    cluster_sync_all();
    if (MODE == kDv && threadIdx.x == 0) pdl_wait();  // the stream's next work follows both
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2u * kAccCols)
                     : "memory");
    }
}

// ------------------------------------------------------------------ dG and dU
// dG = dH U act'(G), dU = dH act(G) (M x ld, ld = N rounded up to 8; the columns past N are
// not written and not read), 8 columns per thread; clears the products' counters as well.
// Memory-bound: 10 bytes an entry.  Rounded to fp16 because they are operands of the products
// that follow (the gradients' relative error against 64 bits is 2.9e-4, 2.1e-4 of it the rounding of
// the result; keeping the remainders would double the products); an overflow becomes an
// infinity there, which a loss scaler looks for.
__global__ void __launch_bounds__(256)
gate_grad_kernel(const uint16_t* __restrict__ G, int ldg, const uint16_t* __restrict__ U, int ldu,
                 const uint16_t* __restrict__ dH, int ldh, int M, int N, int act, int vec,
                 uint16_t* __restrict__ dG, uint16_t* __restrict__ dU, int ld, uint32_t* __restrict__ clear,
                 uint32_t n_clear) {
    pdl_launch_dependents();
    for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < n_clear; i += gridDim.x * blockDim.x) clear[i] = 0u;
    const int per_row = (N + 7) / 8;
    const long long n = (long long)M * per_row;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
        const long long m = i / per_row;
        const int c = 8 * (int)(i - m * per_row);
        uint16_t g[8], u[8], h[8];
        const size_t og = (size_t)m * ldg + c, ou = (size_t)m * ldu + c, oh = (size_t)m * ldh + c;
        if (vec && c + 8 <= N) {
            *(uint4*)g = *(const uint4*)(G + og);
            *(uint4*)u = *(const uint4*)(U + ou);
            *(uint4*)h = *(const uint4*)(dH + oh);
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const bool in = c + e < N;
                g[e] = in ? G[og + e] : 0;
                u[e] = in ? U[ou + e] : 0;
                h[e] = in ? dH[oh + e] : 0;
            }
        }
        uint32_t wg[4], wu[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            float dg[2], du[2];
#pragma unroll
            for (int q = 0; q < 2; q++) {
                const float fh = __half2float(__ushort_as_half(h[2 * e + q]));
                float a, slope;
                act_grad_f32(__half2float(__ushort_as_half(g[2 * e + q])), act, a, slope);
                dg[q] = fh * __half2float(__ushort_as_half(u[2 * e + q])) * slope;
                du[q] = fh * a;
            }
            wg[e] = pack2(dg[0], dg[1]);
            wu[e] = pack2(du[0], du[1]);
        }
        *(uint4*)(dG + (size_t)m * ld + c) = make_uint4(wg[0], wg[1], wg[2], wg[3]);
        *(uint4*)(dU + (size_t)m * ld + c) = make_uint4(wu[0], wu[1], wu[2], wu[3]);
    }
}

// ------------------------------------------------------------------ host side

// SM pairs (clusters of two CTAs with the product's shared memory) of the current device.
int gemm_pairs() {
    static int cache[kMaxDevices];
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    std::lock_guard<std::mutex> lock(mu);
    if (!cache[dev]) {
        const void* fns[4] = {(const void*)gemm_kernel<kEp>, (const void*)gemm_kernel<kFfn>,
                              (const void*)gemm_kernel<kDx>, (const void*)gemm_kernel<kDv>};
        for (const void* f : fns)
            if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) != cudaSuccess) {
                (void)cudaGetLastError();
                return 0;
            }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemLimit;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, gemm_kernel<kEp>, &cfg) != cudaSuccess) n = 0;
        (void)cudaGetLastError();
        cache[dev] = n;
    }
    return cache[dev];
}

struct GemmPlan {
    int m_tiles, n_tiles, problems, BN, parts, stages;
    long long tiles, n_units;
    uint32_t block_bytes, stage_bytes, off_bar, off_stage;
    size_t smem;
    uint64_t counter_bytes, partial_bytes;
    double cost;  // microseconds
};

// Column tile and split of the reduction from a small cost model in microseconds: a step of
// 64 costs 0.36 at BN = 256 and 0.22 at 128, a unit 2 more, a split piece its fp32 partials.
// cols: result columns counted so that a tile holds BN of them (kFfn: 2 N).
int plan_gemm(long long rows, long long cols, int problems, long long ksteps, int pairs, GemmPlan* g) {
    if (pairs <= 0) return SPW_ERR_CUDA;
    double best = 1e300;
    g->problems = problems;
    for (int BN = 256; BN >= 128; BN -= 128) {
        const long long mt = (rows + 255) / 256, nt = (cols + BN - 1) / BN;
        const long long tiles = mt * nt * problems;
        const double step = BN == 256 ? 0.36 : 0.22;
        for (int parts = 1; parts <= 16 && parts * 4 <= (ksteps < 4 ? 4 : ksteps); parts++) {
            const long long units = tiles * parts;
            const double waves = (double)((units + pairs - 1) / pairs);
            const double ks = (double)((ksteps + parts - 1) / parts);
            const double cost = waves * (ks * step + 2.0 + (parts > 1 ? 1.0 + BN * 0.01 * (1 + parts) : 0.0));
            if (cost < best * 0.98) {
                best = cost;
                g->BN = BN;
                g->m_tiles = (int)mt;
                g->n_tiles = (int)nt;
                g->tiles = tiles;
                g->parts = parts;
            }
        }
    }
    if (g->tiles * g->parts > 0x3fffffffll) return SPW_ERR_UNSUPPORTED;
    g->cost = best;
    const long long split = g->parts > 1 ? g->tiles : 0;
    g->n_units = g->tiles * g->parts;
    g->counter_bytes = round_up_u64(8ull * (uint64_t)split, 256);
    g->partial_bytes = 4ull * (uint64_t)split * g->parts * 2 * g->BN * kCtaRows;
    g->block_bytes = kABytes + (uint32_t)g->BN / 2 * 128;
    g->stage_bytes = kStageBlocks * g->block_bytes;
    const uint32_t bars = 8u * (2 * kMaxStages + 5) + 32u;
    const uint32_t blocks = 4u * kEpiWarps * 32 * 33;
    g->stages = (int)((kSmemLimit - 1024 - bars - blocks) / g->stage_bytes);
    if (g->stages > kMaxStages) g->stages = kMaxStages;
    g->off_bar = (uint32_t)g->stages * g->stage_bytes;
    g->off_stage = g->off_bar + (uint32_t)round_up_u64(bars, 16);
    g->smem = (size_t)g->off_stage + blocks + 1024;
    return SPW_OK;
}

void fill_params(const GemmPlan& g, long long ksteps, GemmParams* p) {
    memset(p, 0, sizeof(*p));
    p->m_tiles = g.m_tiles;
    p->n_tiles = g.n_tiles;
    p->group_m = g.m_tiles < 16 ? g.m_tiles : 16;
    p->problem_tiles = g.m_tiles * g.n_tiles;
    p->n_units = (int)g.n_units;
    p->parts = g.parts;
    p->ksteps = p->kseg = (int)ksteps;
    p->BN = g.BN;
    p->stages = g.stages;
    p->block_bytes = g.block_bytes;
    p->stage_bytes = g.stage_bytes;
    p->off_bar = g.off_bar;
    p->off_stage = g.off_stage;
    p->wait_limit = wait_limit_cycles();
    p->status = device_status_ptr();
}

// early: may start while the kernel before it, of the same call, still runs.
template <int MODE>
int launch_gemm(const GemmPlan& g, const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b0,
                const CUtensorMap& b1, const GemmParams& p, int pairs, bool early, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    const long long n = g.n_units < pairs ? g.n_units : pairs;
    cfg.gridDim = dim3((unsigned)(2 * n));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = g.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 2 : 1;
    SPW_CUDA_TRY(cudaLaunchKernelEx(&cfg, gemm_kernel<MODE>, a0, a1, b0, b1, p));
    return SPW_OK;
}

int ktp_of(const spw_format* h) { return (int)round_up_u64(h->n_ktiles, 4); }

uint64_t dense_bytes(const spw_format* h) {
    return round_up_u64(h->n_strips, 4) * (uint64_t)ktp_of(h) * 8192;
}

// Expands one or two weights into blocks of `strips` strips, and clears counters.
int expand(int n, const spw_format* const* hdrs, const void* const* bufs, uint16_t* const* outs, int strips, void* clear,
           uint64_t clear_bytes, cudaStream_t s) {
    ExpandParams p;
    memset(&p, 0, sizeof(p));
    p.clear = (uint32_t*)clear;
    p.n_clear = (uint32_t)(clear_bytes / 4);
    p.strips = strips;
    p.ktp = ktp_of(hdrs[0]);
    uint32_t units = 0;
    for (int l = 0; l < n; l++) {
        const spw_format& h = *hdrs[l];
        const uint8_t* buf = (const uint8_t*)bufs[l];
        ExpandLayer& L = p.L[l];
        L.bitmaps = (const uint64_t*)(buf + h.off_bitmaps);
        L.tileptr = (const uint32_t*)(buf + h.off_tileptr);
        L.values = (const uint16_t*)(buf + h.off_values);
        L.values_units = (h.bytes_total - h.off_values) / 16;
        L.max_units = h.max_tile_units;
        L.out = outs[l];
        L.n_ktiles = (int)h.n_ktiles;
        L.n_tiles = (long long)h.n_strips * h.n_ktiles;
        p.tiles += L.n_tiles;
        if (h.max_tile_units > units) units = h.max_tile_units;
    }
    p.status = device_status_ptr();
    if (!p.status) return SPW_ERR_CUDA;
    p.warp_smem = kRecBytes + 16u * units + 32u;  // slack before and after the values
    const size_t smem = (size_t)kExpandWarps * p.warp_smem;
    if (smem > 48 * 1024)
        SPW_CUDA_TRY(cudaFuncSetAttribute(expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (int)(kExpandWarps * (kRecBytes + 16u * 512u + 32u))));
    const int per_sm = smem > 0 ? (int)((size_t)kSmemLimit / (smem + 1024)) : 8;
    const long long want = (p.tiles + kExpandWarps - 1) / kExpandWarps;
    const long long most = (long long)device_sm_count() * (per_sm < 1 ? 1 : per_sm > 8 ? 8 : per_sm);
    if (most <= 0) return SPW_ERR_CUDA;
    const long long grid = want < most ? want : most;
    expand_kernel<<<(unsigned)grid, 32 * kExpandWarps, smem, s>>>(p);
    SPW_LAUNCH_CHECK();
    return SPW_OK;
}

// Row stride in bytes for a tensor map: a single row may have any leading dimension.
uint64_t map_ld(int ld, int rows) { return 2ull * (rows > 1 ? (uint64_t)ld : round_up_u64((uint64_t)ld, 8)); }


// Workspace sections: the split counters of each product, the expanded weights, dG and dU
// where there are any, and the fp32 partials.  They start at the workspace's first multiple of
// kWsAlign (the expansion stores 32 bytes at a time, and the caller's pointer need only be a
// multiple of 16), so `total` holds what that may skip.
constexpr uint64_t kWsAlign = 256;
struct Layout {
    GemmPlan fwd, dx, dv;
    bool fwd_direct, dx_direct;  // by the direct form (spmm_direct.cu): no workspace
    uint64_t dv_counters, dv_partials, counters, dense, grads, partials, total;  // counters: the bytes to clear
    int ldn;
};

constexpr int kForward = 1, kDxOut = 2, kDvOut = 4;

// Whether the direct form takes less time than expansion and product.  Measured: the expansion
// takes 3.5 us and 0.53 us for a million entries, the product 3 us beside its units and 0.17 for a
// million entries (what L2 does not keep), and the clearing of counters 2.  (Direct / expanded:
// 4096 x 4096 with an epilogue 23 / 32 us at 256 tokens, 32 / 33 at 512, 47 / 43 at 1024; gated,
// 11008 x 4096, 110 / 122 at 256, 137 / 148 at 512, 182 / 168 at 700.)
bool choose_direct(int mode, const spw_format* h, const spw_format* h2, int M, const GemmPlan& g) {
    const double entries = (h2 ? 2.0 : 1.0) * h->n_strips * (double)h->n_ktiles * kStripRows * kTileCols;
    const double other = g.cost + 6.5 + entries * 0.7e-6 + (g.counter_bytes ? 2.0 : 0.0);
    const double direct = direct_cost(mode, h, h2, M);
    return direct >= 0.0 && direct <= other;
}

// h2: the second weight's header, or null.
int make_layout(const spw_format* h, const spw_format* h2, int M, int what, Layout* L) {
    if (M > kMaxDim || h->N > kMaxDim || h->K > kMaxDim) return SPW_ERR_UNSUPPORTED;
    const int pairs = gemm_pairs();
    const int weights = h2 ? 2 : 1;
    memset(L, 0, sizeof(*L));
    L->ldn = (int)round_up_u64(h->N, 8);
    uint64_t c = 0, part = 0, dense = 0;
    int rc;
    if (what & kForward) {
        rc = plan_gemm(M, (long long)weights * h->N, 1, h->n_ktiles, pairs, &L->fwd);
        if (rc != SPW_OK) return rc;
        L->fwd_direct = choose_direct(h2 ? kFfn : kEp, h, h2, M, L->fwd);
        if (!L->fwd_direct) {
            c = L->fwd.counter_bytes;
            part = L->fwd.partial_bytes;
            dense = (uint64_t)weights * dense_bytes(h);
        }
    }
    if (what & kDxOut) {
        rc = plan_gemm(M, h->K, 1, (long long)weights * h->n_strips, pairs, &L->dx);
        if (rc != SPW_OK) return rc;
        L->dx_direct = choose_direct(kDx, h, h2, M, L->dx);
        if (!L->dx_direct) {
            c += L->dx.counter_bytes;
            if (L->dx.partial_bytes > part) part = L->dx.partial_bytes;
            dense = (uint64_t)weights * dense_bytes(h);
        }
    }
    L->dv_counters = c;
    if (what & kDvOut) {
        rc = plan_gemm(h->N, h->K, weights, ((long long)M + 63) / 64, pairs, &L->dv);
        if (rc != SPW_OK) return rc;
        c += L->dv.counter_bytes;
        L->dv_partials = part;  // beside those of dX: the two may run at the same time
        part += L->dv.partial_bytes;
    }
    L->counters = c;
    L->dense = c;
    L->grads = L->dense + dense;
    const uint64_t grads =
        weights == 2 && (what & (kDxOut | kDvOut)) ? 2 * round_up_u64(2ull * (uint64_t)M * L->ldn, 256) : 0;
    L->partials = L->grads + grads;
    L->total = L->partials + part;
    if (L->total) L->total += kWsAlign - 16;
    return SPW_OK;
}

// Where the sections of a checked workspace start (null stays null: nothing is read then).
uint8_t* ws_base(void* d_ws) { return (uint8_t*)(((uintptr_t)d_ws + kWsAlign - 1) & ~(uintptr_t)(kWsAlign - 1)); }

int check_ws(const void* d_ws, uint64_t ws_bytes, const Layout& L) {
    if (!L.total) return SPW_OK;
    if (!d_ws) return SPW_ERR_INVALID_ARG;
    if (ws_bytes < L.total) return SPW_ERR_BUFFER_TOO_SMALL;
    if (!aligned16(d_ws)) return SPW_ERR_ALIGNMENT;
    return SPW_OK;
}

// A forward product (kEp: one weight; kFfn: gate and up) by the form that the layout chose.
template <int MODE>
int run_forward(const Layout& L, const spw_format* const* hdrs, const void* const* bufs, const uint16_t* X, int M, int ldx,
                const PrefillOut& o, uint8_t* ws, cudaStream_t s) {
    constexpr int kWeights = MODE == kFfn ? 2 : 1;
    const spw_format* h = hdrs[0];
    if (L.fwd_direct) {
        DirectCall c;
        memset(&c, 0, sizeof(c));
        c.mode = MODE;
        for (int w = 0; w < kWeights; w++) {
            c.h[w] = hdrs[w];
            c.buf[w] = bufs[w];
        }
        c.x[0] = X;
        c.ldx_bytes[0] = map_ld(ldx, M);
        c.M = M;
        c.out = o;
        return direct_launch(c, s);
    }
    const GemmPlan& g = L.fwd;
    CUtensorMap a, b[2];
    uint16_t* dense[2];
    int rc = encode_map_f16(&a, X, h->K, (uint64_t)M, map_ld(ldx, M), kBK, kCtaRows);
    for (int w = 0; w < kWeights && rc == SPW_OK; w++) {
        dense[w] = (uint16_t*)(ws + L.dense + (uint64_t)w * dense_bytes(h));
        rc = encode_map_f16(&b[w], dense[w], 64, dense_bytes(h) / 128, 128, 64, (uint32_t)g.BN / 2, false);
    }
    if (rc != SPW_OK) return rc;
    GemmParams p;
    fill_params(g, h->n_ktiles, &p);
    if (!p.status) return SPW_ERR_CUDA;
    p.o = o;
    p.ktp = ktp_of(h);
    p.counters = (uint32_t*)ws;
    p.partials = (float*)(ws + L.partials);
    rc = expand(kWeights, hdrs, bufs, dense, g.BN / 128, ws, L.counters, s);
    if (rc != SPW_OK) return rc;
    return launch_gemm<MODE>(g, a, a, b[0], b[kWeights - 1], p, gemm_pairs(), true, s);
}

// dX = sum over the weights of dY_w W_w, by the form that the layout chose.
int run_dx(const spw_format* const* hdrs, const void* const* bufs, int weights, const Layout& L, uint8_t* ws,
           uint32_t* counters, const uint16_t* const* dY, const uint64_t* ld_bytes, int M, uint16_t* dX, int lddx,
           bool early, cudaStream_t s) {
    const GemmPlan& g = L.dx;
    const spw_format* h = hdrs[0];
    PrefillOut o;
    memset(&o, 0, sizeof(o));
    o.rows = M;
    o.cols = (int)h->K;
    o.Y = dX;
    o.ldy = lddx;
    o.vec = vec_bits(o);
    if (L.dx_direct) {
        DirectCall c;
        memset(&c, 0, sizeof(c));
        c.mode = kDx;
        for (int w = 0; w < weights; w++) {
            c.h[w] = hdrs[w];
            c.buf[w] = bufs[w];
            c.x[w] = dY[w];
            c.ldx_bytes[w] = ld_bytes[w];
        }
        c.M = M;
        c.out = o;
        c.early = early;
        return direct_launch(c, s);
    }
    uint16_t* dense[2];
    for (int w = 0; w < weights; w++) dense[w] = (uint16_t*)(ws + L.dense + (uint64_t)w * dense_bytes(h));
    const int erc = expand(weights, hdrs, bufs, dense, 1, nullptr, 0, s);
    if (erc != SPW_OK) return erc;
    CUtensorMap a[2], b[2];
    for (int w = 0; w < weights; w++) {
        int rc = encode_map_f16(&a[w], dY[w], h->N, (uint64_t)M, ld_bytes[w], kBK, kCtaRows);
        if (rc != SPW_OK) return rc;
        rc = encode_map_f16(&b[w], ws + L.dense + w * dense_bytes(h), 64, dense_bytes(h) / 128, 128, 64,
                            (uint32_t)g.BN / 2, false);
        if (rc != SPW_OK) return rc;
    }
    if (weights == 1) {
        a[1] = a[0];
        b[1] = b[0];
    }
    GemmParams p;
    fill_params(g, (long long)weights * h->n_strips, &p);
    if (!p.status) return SPW_ERR_CUDA;
    p.kseg = (int)h->n_strips;
    p.ktp = ktp_of(h);
    p.o = o;
    p.counters = counters;
    p.partials = (float*)(ws + L.partials);
    return launch_gemm<kDx>(g, a[0], a[1], b[0], b[1], p, gemm_pairs(), true, s);
}

// Gradients of the kept weights, dY_w^T X at their positions, packed as the values are.
int run_dv(const spw_format* const* hdrs, const void* const* bufs, int weights, const Layout& L, uint8_t* ws,
           uint32_t* counters, const uint16_t* const* dY, const uint64_t* ld_bytes, const uint16_t* X, int ldx, int M,
           uint16_t* const* dV, bool early, cudaStream_t s) {
    const GemmPlan& g = L.dv;
    const spw_format* h = hdrs[0];
    CUtensorMap a[2], b;
    int rc = encode_map_f16(&b, X, h->K, (uint64_t)M, map_ld(ldx, M), 64, kBK);
    if (rc != SPW_OK) return rc;
    GemmParams p;
    fill_params(g, ((long long)M + 63) / 64, &p);
    if (!p.status) return SPW_ERR_CUDA;
    for (int w = 0; w < weights; w++) {
        rc = encode_map_f16(&a[w], dY[w], h->N, (uint64_t)M, ld_bytes[w], 64, kBK);
        if (rc != SPW_OK) return rc;
        const uint8_t* buf = (const uint8_t*)bufs[w];
        p.bitmaps[w] = (const uint64_t*)(buf + hdrs[w]->off_bitmaps);
        p.tileptr[w] = (const uint32_t*)(buf + hdrs[w]->off_tileptr);
        p.values_units[w] = (hdrs[w]->bytes_total - hdrs[w]->off_values) / 16;
        p.dv[w] = dV[w];
    }
    if (weights == 1) a[1] = a[0];
    p.n_strips = (int)h->n_strips;
    p.n_ktiles = (int)h->n_ktiles;
    p.o.rows = (int)h->N;
    p.o.cols = (int)h->K;
    p.counters = counters;
    p.partials = (float*)(ws + L.partials + L.dv_partials);
    return launch_gemm<kDv>(g, a[0], a[1], b, b, p, gemm_pairs(), early, s);
}

}  // namespace

int vec_bits(const PrefillOut& o) {
    auto ok = [](const void* p, int ld) { return !p || ld % 8 == 0; };
    return (ok(o.Y, o.ldy) ? 1 : 0) | (ok(o.residual, o.ldr) ? 2 : 0) | (ok(o.G, o.ldg) ? 4 : 0) | (ok(o.U, o.ldu) ? 8 : 0) |
           (o.ldy % 2 == 0 && (!o.residual || o.ldr % 2 == 0) ? 16 : 0) | (o.ldg % 2 == 0 ? 32 : 0) |
           (o.ldu % 2 == 0 ? 64 : 0);
}

// Checks of an epilogue's arguments for a result of N columns.
int check_epilogue(const spw_epilogue* ep, int N) {
    if (!ep) return SPW_OK;
    if (!act_ok(ep->act) || (ep->residual && ep->ldr < N)) return SPW_ERR_INVALID_ARG;
    if (!aligned16(ep->bias) || !aligned16(ep->residual)) return SPW_ERR_ALIGNMENT;
    return SPW_OK;
}

}  // namespace spw

using namespace spw;

extern "C" {

uint64_t spw_spmm_ep_workspace_bytes(const spw_format* hdr, int M) {
    Layout L;
    if (check_header(hdr) != SPW_OK || M < 1 || make_layout(hdr, nullptr, M, kForward, &L) != SPW_OK) return 0;
    return L.total;
}

int spw_spmm_ep(const spw_format* hdr, const void* d_buf, const uint16_t* d_X, int M, int ldx, const spw_epilogue* ep,
                uint16_t* d_Y, int ldy, void* d_ws, uint64_t ws_bytes, void* stream) {
    int rc = check_header(hdr);
    if (rc != SPW_OK) return rc;
    if (M < 0) return SPW_ERR_INVALID_ARG;
    const int N = (int)hdr->N;
    rc = check_epilogue(ep, N);
    if (rc != SPW_OK || M == 0) return rc;
    if (!d_buf || !d_X || !d_Y) return SPW_ERR_INVALID_ARG;
    if (!ld_ok(ldx, (int)hdr->K, M) || ldy < N) return SPW_ERR_INVALID_ARG;
    if (!aligned16(d_buf) || !aligned16(d_X) || !aligned16(d_Y)) return SPW_ERR_ALIGNMENT;
    Layout L;
    rc = make_layout(hdr, nullptr, M, kForward, &L);
    if (rc == SPW_OK) rc = check_ws(d_ws, ws_bytes, L);
    if (rc != SPW_OK) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    PrefillOut o;
    memset(&o, 0, sizeof(o));
    o.rows = M;
    o.cols = N;
    o.Y = d_Y;
    o.ldy = ldy;
    if (ep) {
        o.bias = ep->bias;
        o.act = ep->act;
        o.residual = ep->residual;
        o.ldr = ep->ldr;
    }
    o.vec = vec_bits(o);
    return run_forward<kEp>(L, &hdr, &d_buf, d_X, M, ldx, o, ws_base(d_ws), s);
}

static int check_ffn_pair(const spw_format* hg, const spw_format* hu) {
    int rc = check_header(hg);
    if (rc == SPW_OK) rc = check_header(hu);
    if (rc != SPW_OK) return rc;
    return hg->N == hu->N && hg->K == hu->K ? SPW_OK : SPW_ERR_INVALID_ARG;
}

uint64_t spw_spmm_ffn_workspace_bytes(const spw_format* hdr_gate, const spw_format* hdr_up, int M) {
    Layout L;
    if (check_ffn_pair(hdr_gate, hdr_up) != SPW_OK || M < 1 || make_layout(hdr_gate, hdr_up, M, kForward, &L) != SPW_OK)
        return 0;
    return L.total;
}

int spw_spmm_ffn(const spw_format* hdr_gate, const void* d_buf_gate, const spw_format* hdr_up, const void* d_buf_up,
                 const uint16_t* d_X, int M, int ldx, int act, uint16_t* d_H, int ldh, uint16_t* d_G, int ldg,
                 uint16_t* d_U, int ldu, void* d_ws, uint64_t ws_bytes, void* stream) {
    int rc = check_ffn_pair(hdr_gate, hdr_up);
    if (rc != SPW_OK) return rc;
    if (M < 0 || !act_ok(act) || (d_G == nullptr) != (d_U == nullptr)) return SPW_ERR_INVALID_ARG;
    if (M == 0) return SPW_OK;
    const int N = (int)hdr_gate->N, K = (int)hdr_gate->K;
    if (!d_buf_gate || !d_buf_up || !d_X || !d_H) return SPW_ERR_INVALID_ARG;
    if (!ld_ok(ldx, K, M) || ldh < N || (d_G && (ldg < N || ldu < N))) return SPW_ERR_INVALID_ARG;
    if (!aligned16(d_buf_gate) || !aligned16(d_buf_up) || !aligned16(d_X) || !aligned16(d_H) || !aligned16(d_G) ||
        !aligned16(d_U))
        return SPW_ERR_ALIGNMENT;
    if (d_G && (d_G == d_U || d_G == d_H || d_U == d_H)) return SPW_ERR_INVALID_ARG;
    Layout L;
    rc = make_layout(hdr_gate, hdr_up, M, kForward, &L);
    if (rc == SPW_OK) rc = check_ws(d_ws, ws_bytes, L);
    if (rc != SPW_OK) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    PrefillOut o;
    memset(&o, 0, sizeof(o));
    o.rows = M;
    o.cols = N;
    o.Y = d_H;
    o.ldy = ldh;
    o.G = d_G;
    o.ldg = ldg;
    o.U = d_U;
    o.ldu = ldu;
    o.act = act;
    o.vec = vec_bits(o);
    const spw_format* hdrs[2] = {hdr_gate, hdr_up};
    const void* bufs[2] = {d_buf_gate, d_buf_up};
    return run_forward<kFfn>(L, hdrs, bufs, d_X, M, ldx, o, ws_base(d_ws), s);
}

uint64_t spw_spmm_ffn_backward_workspace_bytes(const spw_format* hdr_gate, const spw_format* hdr_up, int M) {
    Layout L;
    if (check_ffn_pair(hdr_gate, hdr_up) != SPW_OK || M < 1 ||
        make_layout(hdr_gate, hdr_up, M, kDxOut | kDvOut, &L) != SPW_OK)
        return 0;
    return L.total;
}

int spw_spmm_ffn_backward(const spw_format* hdr_gate, const void* d_buf_gate, const spw_format* hdr_up,
                          const void* d_buf_up, const uint16_t* d_X, int M, int ldx, int act, const uint16_t* d_G,
                          int ldg, const uint16_t* d_U, int ldu, const uint16_t* d_dH, int lddh, uint16_t* d_dX,
                          int lddx, uint16_t* d_dV_gate, uint16_t* d_dV_up, void* d_ws, uint64_t ws_bytes,
                          void* stream) {
    int rc = check_ffn_pair(hdr_gate, hdr_up);
    if (rc != SPW_OK) return rc;
    if (M < 0 || !act_ok(act) || (d_dV_gate == nullptr) != (d_dV_up == nullptr)) return SPW_ERR_INVALID_ARG;
    const int N = (int)hdr_gate->N, K = (int)hdr_gate->K;
    if (!aligned16(d_buf_gate) || !aligned16(d_buf_up) || !aligned16(d_X) || !aligned16(d_G) || !aligned16(d_U) ||
        !aligned16(d_dH) || !aligned16(d_dX) || !aligned16(d_dV_gate) || !aligned16(d_dV_up))
        return SPW_ERR_ALIGNMENT;
    // (with nothing kept a gradient has no entries, and any address stands for it)
    if (d_dV_gate && d_dV_gate == d_dV_up && hdr_gate->bytes_total > hdr_gate->off_values &&
        hdr_up->bytes_total > hdr_up->off_values)
        return SPW_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (M == 0) {  // no token: the kept weights' gradient is zero
        if (d_dV_gate) {
            SPW_CUDA_TRY(cudaMemsetAsync(d_dV_gate, 0, hdr_gate->bytes_total - hdr_gate->off_values, s));
            SPW_CUDA_TRY(cudaMemsetAsync(d_dV_up, 0, hdr_up->bytes_total - hdr_up->off_values, s));
        }
        return SPW_OK;
    }
    if (!d_dX && !d_dV_gate) return SPW_ERR_INVALID_ARG;
    if (!d_buf_gate || !d_buf_up || !d_G || !d_U || !d_dH || (d_dV_gate && !d_X)) return SPW_ERR_INVALID_ARG;
    if (ldg < N || ldu < N || lddh < N || (d_dX && lddx < K) || (d_dV_gate && !ld_ok(ldx, K, M)))
        return SPW_ERR_INVALID_ARG;
    Layout L;
    rc = make_layout(hdr_gate, hdr_up, M, kDxOut | kDvOut, &L);
    if (rc == SPW_OK) rc = check_ws(d_ws, ws_bytes, L);
    if (rc != SPW_OK) return rc;
    uint8_t* ws = ws_base(d_ws);
    uint16_t* dG = (uint16_t*)(ws + L.grads);
    uint16_t* dU = (uint16_t*)(ws + L.grads + round_up_u64(2ull * (uint64_t)M * L.ldn, 256));
    const long long n = (long long)M * ((N + 7) / 8);
    const long long most = 16ll * device_sm_count();
    if (most <= 0) return SPW_ERR_CUDA;
    const long long grid = (n + 255) / 256 < most ? (n + 255) / 256 : most;
    const int vec = ldg % 8 == 0 && ldu % 8 == 0 && lddh % 8 == 0 ? 1 : 0;
    gate_grad_kernel<<<(unsigned)grid, 256, 0, s>>>(d_G, ldg, d_U, ldu, d_dH, lddh, M, N, act, vec, dG, dU, L.ldn,
                                                    (uint32_t*)ws, (uint32_t)(L.counters / 4));
    SPW_LAUNCH_CHECK();
    const spw_format* hdrs[2] = {hdr_gate, hdr_up};
    const void* bufs[2] = {d_buf_gate, d_buf_up};
    const uint16_t* dY[2] = {dG, dU};
    const uint64_t ld_bytes[2] = {2ull * L.ldn, 2ull * L.ldn};
    uint32_t* counters = (uint32_t*)ws;
    if (d_dX) {
        rc = run_dx(hdrs, bufs, 2, L, ws, counters, dY, ld_bytes, M, d_dX, lddx, true, s);
        if (rc != SPW_OK) return rc;
    }
    if (d_dV_gate) {
        uint16_t* dV[2] = {d_dV_gate, d_dV_up};
        rc = run_dv(hdrs, bufs, 2, L, ws, counters + L.dv_counters / 4, dY, ld_bytes, d_X, ldx, M, dV, d_dX != nullptr, s);
    }
    return rc;
}

uint64_t spw_spmm_backward_workspace_bytes(const spw_format* hdr, int M) {
    Layout L;
    if (check_header(hdr) != SPW_OK || M < 1 || make_layout(hdr, nullptr, M, kDxOut | kDvOut, &L) != SPW_OK) return 0;
    return L.total;
}

int spw_spmm_backward(const spw_format* hdr, const void* d_buf, const uint16_t* d_X, int M, int ldx,
                      const uint16_t* d_dY, int lddy, uint16_t* d_dX, int lddx, uint16_t* d_dV, void* d_ws,
                      uint64_t ws_bytes, void* stream) {
    int rc = check_header(hdr);
    if (rc != SPW_OK) return rc;
    if (M < 0) return SPW_ERR_INVALID_ARG;
    const int N = (int)hdr->N, K = (int)hdr->K;
    if (!aligned16(d_buf) || !aligned16(d_X) || !aligned16(d_dY) || !aligned16(d_dX) || !aligned16(d_dV))
        return SPW_ERR_ALIGNMENT;
    cudaStream_t s = (cudaStream_t)stream;
    if (M == 0) {
        if (d_dV) SPW_CUDA_TRY(cudaMemsetAsync(d_dV, 0, hdr->bytes_total - hdr->off_values, s));
        return SPW_OK;
    }
    if (!d_dX && !d_dV) return SPW_ERR_INVALID_ARG;
    if (!d_buf || !d_dY || (d_dV && !d_X)) return SPW_ERR_INVALID_ARG;
    if (!ld_ok(lddy, N, M) || (d_dX && lddx < K) || (d_dV && !ld_ok(ldx, K, M))) return SPW_ERR_INVALID_ARG;
    Layout L;
    rc = make_layout(hdr, nullptr, M, kDxOut | kDvOut, &L);
    if (rc == SPW_OK) rc = check_ws(d_ws, ws_bytes, L);
    if (rc != SPW_OK) return rc;
    uint8_t* ws = ws_base(d_ws);
    uint32_t* counters = (uint32_t*)ws;
    const uint64_t ld_bytes[1] = {map_ld(lddy, M)};
    if (L.counters) SPW_CUDA_TRY(cudaMemsetAsync(ws, 0, L.counters, s));
    if (d_dX) {
        rc = run_dx(&hdr, &d_buf, 1, L, ws, counters, &d_dY, ld_bytes, M, d_dX, lddx, false, s);
        if (rc != SPW_OK) return rc;
    }
    if (d_dV)
        rc = run_dv(&hdr, &d_buf, 1, L, ws, counters + L.dv_counters / 4, &d_dY, ld_bytes, d_X, ldx, M, &d_dV, d_dX != nullptr, s);
    return rc;
}

}  // extern "C"
