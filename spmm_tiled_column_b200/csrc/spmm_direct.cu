// spmm_direct.cu -- the prefill products with an epilogue for few tokens: the compressed
// weight is decoded into shared memory as the MMA's A operand and never written out dense.
//
//   kEp   Y = act(X W^T + bias) + residual     A = 128 weight rows (two strips)
//   kFfn  H = act(X Wg^T) * (X Wu^T)           A = 64 gate rows, then the same 64 up rows
//   kDx   dX = sum over the weights of dY W    A = 128 weight columns (two k-tiles), MN-major
//   kDecode  as kEp for at most 16 rows, with the decode's threshold rule or column set
//
// With few tokens each weight tile is needed once or twice, so what bounds the product is the
// decoding (for a 64 x 64 tile about 900 warp instructions and, the exchange of the pieces
// included, 507 shared-memory wavefronts: 11008 x 4096 at 128 tokens; an SM does two tiles in
// 0.58 us) and, for small weights, the latency of the chain pointers ->
// compressed tile -> decode -> MMA -> result (6.3 us for one tile).  At 50 %: 4096 x 4096 with an
// epilogue 16.2 us at 16 tokens, 19.2 at 128; 4096 x 11008 32 and 36; 11008 x 4096 gated 66 and 77.
// The design follows from that:
//   * A CTA computes 128 x MT (MT tokens, at most 512; fp32 accumulator in tensor memory)
//     over one of `parts` pieces of the reduction; the pieces of a tile form a cluster, which
//     adds them through distributed shared memory: no workspace, no counters, every CTA of the
//     cluster finishes its share of the tokens.  Summed in piece order (deterministic).
//   * Decoders work in groups of four warps, each group on a step (two 64 x 64 tiles) of its
//     own, a warp on 32 columns of one tile: the waits, scans and look-ups of the groups
//     overlap.  A CTA has four groups, or two where two such CTAs an SM fit the grid better.
//     A step's dense tiles are stored as core matrices of 8 rows x 16 bytes (no swizzle),
//     which the MMA takes K-major (kEp, kFfn) or MN-major (kDx) from the same bytes.
//   * warp 0: TMA of the token tiles (kDecode: loads them itself and applies the rule on the
//     way into shared memory); warp 1: MMAs; warp 2: tile pointers (16 steps at a time,
//     ahead) and bulk copies of the compressed tiles; warps 3..: decoders.
//   * The result goes through shared memory, so a warp stores whole rows of 128 (kFfn: 64)
//     neighbouring columns.
// Barriers and records of a ring are indexed n % kRing with kRing a multiple of the groups, so
// that no wait by parity runs a whole phase ahead; memory slots are n % (slots).  Every wait is
// bounded and polls the CTA's abort flag; the cluster barriers are passed on an abort too.
#include <string.h>

#include <mutex>

#include "spw_prefill.cuh"
#include "spw_tcgen05.cuh"

namespace spw {
namespace {

constexpr int kBK = 64;
constexpr int kRing = 8;
constexpr uint32_t kWBytes = 128 * kBK * 2;  // a step's dense tiles, 16 KB
constexpr uint32_t kRecBytes = 528;          // a decoder warp's records: 32 low halves, 32 high ones
constexpr int kSmemLimit = 227 * 1024;
constexpr int kFirstDecoder = 3;
constexpr int kMaxParts = 8;
constexpr int kMaxTok = 512;

__host__ __device__ constexpr int threads_of(int groups) { return 32 * (kFirstDecoder + 4 * groups); }

struct DirectLayer {
    const uint64_t* bitmaps;
    const uint32_t* tileptr;
    const uint16_t* values;
    uint64_t values_units;  // the values section, in 16-byte units
};

struct DirectParams {
    DirectLayer L[2];
    PrefillOut o;
    int n_strips, n_ktiles;
    int steps, seg;             // of the reduction; of its first segment (kDx)
    int parts, m_tiles, MT, nh; // nh MMAs of MT / nh tokens a slice
    int n_acc;                  // accumulators: 4 for few tokens, where a chain of MMAs waits for its own results
    int sx, sw, sr;             // slots of token tiles, dense tiles, compressed tiles
    int chunk;                  // tokens of the result that shared memory holds at a time
    uint32_t x_bytes, val_slot, raw_bytes, tmem_cols;
    uint32_t off_w, off_raw, off_rec, off_bar;
    int* status;
    long long wait_limit;
    // kDecode: the rows, the rule
    const uint16_t* x;
    const uint32_t* act_bits;
    int B, K, ldx;
    uint32_t t_bits;  // magnitude bits of the smallest fp16 not below the threshold, at least 1
};

__device__ inline float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Four values to columns col .. col+3 of a row (vec: 8-byte accesses are allowed).
__device__ inline void store4(uint16_t* row, int col, int cols, bool vec, const float (&v)[4]) {
    if (vec && col + 4 <= cols) {
        const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
        *(uint2*)(row + col) = make_uint2(*(const uint32_t*)&a, *(const uint32_t*)&b);
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (col + e < cols) row[col + e] = __half_as_ushort(__float2half_rn(v[e]));
    }
}
__device__ inline void add4(const uint16_t* row, int col, int cols, bool vec, float (&v)[4]) {
    if (vec && col + 4 <= cols) {
        const uint2 r = *(const uint2*)(row + col);
        const float2 a = __half22float2(*(const __half2*)&r.x), b = __half22float2(*(const __half2*)&r.y);
        v[0] += a.x;
        v[1] += a.y;
        v[2] += b.x;
        v[3] += b.y;
    } else {
#pragma unroll
        for (int e = 0; e < 4; e++)
            if (col + e < cols) v[e] += __half2float(__ushort_as_half(row[col + e]));
    }
}

// Tile q of step k of the weight tile wt: weight, strip and k-tile; strip < 0: outside.
struct TileAt {
    int w, strip, kt;
};
template <int MODE>
__device__ inline TileAt tile_at(const DirectParams& p, int wt, int k, int q) {
    TileAt t;
    if constexpr (MODE == kDx) {
        t.w = k >= p.seg ? 1 : 0;
        t.strip = k - t.w * p.seg;
        t.kt = 2 * wt + q;
        if (t.kt >= p.n_ktiles) t.strip = -1;
    } else {
        t.w = MODE == kFfn ? q : 0;
        t.strip = MODE == kFfn ? wt : 2 * wt + q;
        t.kt = k;
        if (t.strip >= p.n_strips) t.strip = -1;
    }
    return t;
}

template <int MODE, int GROUPS>
__global__ void __launch_bounds__(threads_of(GROUPS), GROUPS == 2 ? 2 : 1)
direct_kernel(const __grid_constant__ CUtensorMap tx0, const __grid_constant__ CUtensorMap tx1,
              const __grid_constant__ DirectParams p) {
    constexpr int kThreads = threads_of(GROUPS);
    static_assert(kRing % GROUPS == 0, "");
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = p.parts > 1 ? (int)cluster_rank() : 0;
    const int tile = (int)blockIdx.x / p.parts;
    const int wt = tile / p.m_tiles, mt = tile - wt * p.m_tiles;
    const int m0 = mt * p.MT;
    const int k0 = (int)((long long)part * p.steps / p.parts);
    const int nk = (int)((long long)(part + 1) * p.steps / p.parts) - k0;

    uint64_t* x_full = (uint64_t*)(smem + p.off_bar);
    uint64_t* x_empty = x_full + kRing;
    uint64_t* r_full = x_empty + kRing;
    uint64_t* r_empty = r_full + kRing;
    uint64_t* w_full = r_empty + kRing;
    uint64_t* w_empty = w_full + kRing;
    uint64_t* acc_full = w_empty + kRing;
    uint64_t* drain = acc_full + 1;
    uint32_t* r_info = (uint32_t*)(drain + 1);  // units of a step's two tiles (~0: not to be decoded)
    uint32_t* tmem_slot = r_info + 2 * kRing;
    volatile int* abort_flag = (volatile int*)(tmem_slot + 1);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; i++) {
            mbar_init(smem_u32(&x_full[i]), 1);
            mbar_init(smem_u32(&x_empty[i]), 1);
            mbar_init(smem_u32(&r_full[i]), 2);
            mbar_init(smem_u32(&r_empty[i]), 4);
            mbar_init(smem_u32(&w_full[i]), 4);
            mbar_init(smem_u32(&w_empty[i]), 1);
        }
        mbar_init(smem_u32(acc_full), 1);
        mbar_init(smem_u32(drain), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(p.tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // Raw producer: lane (j, q) = (lane / 2, lane % 2) holds where tile q of step base + j starts
    // and ends.  The first look-up is on its way while the barriers are set up.
    uint32_t u0 = 0, u1 = 0;
    auto pointers = [&](int base) {
        const int i = base + (lane >> 1);
        u0 = u1 = 0;
        if (i >= nk) return;
        const TileAt t = tile_at<MODE>(p, wt, k0 + i, lane & 1);
        if (t.strip < 0) return;
        const uint32_t* at = p.L[t.w].tileptr + (size_t)t.strip * p.n_ktiles + t.kt;
        u0 = __ldg(at);
        u1 = __ldg(at + 1);
    };
    if (warp == 2) pointers(0);
    if (MODE != kDecode && warp == 0 && lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tx0) : "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int tok = p.MT / p.nh;  // tokens of an MMA

    // kDx may have been launched while the kernel that writes dG and dU still runs: warp 0, which
    // alone reads them, waits for its end, then lets the next kernel of the call start.
    int x_issued = 0, r_issued = 0;
    if (warp == 0) {
        if constexpr (MODE == kDx) {
            pdl_wait();
            pdl_launch_dependents();
        }
        if constexpr (MODE == kDecode) {
            // Rows with the rule applied, written where TMA would put them (128-byte swizzle).  A
            // lane has four 16-byte chunks of the 16 x 64 tile: rows lane / 8 + 4 i, columns 8 c ..
            // On fp16 values |v| < t is a comparison of magnitude bits with those of the smallest
            // fp16 not below t (p.t_bits, at least 1: an exact zero is dropped, NaN is kept); with
            // the sign bits set, two subtractions in one word borrow nothing from each other.
            const int c = lane & 7, r0 = lane >> 3;
            const uint32_t tb = p.t_bits | p.t_bits << 16;
            // Two steps at a time under one proxy fence, the next two on their way meanwhile.
            uint4 v[2][4];
            uint32_t on[2] = {0xFFu, 0xFFu};
            auto fetch = [&](int k, uint4 (&to)[4], uint32_t& bits) {
                const int col = kBK * k + 8 * c;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int r = r0 + 4 * i;
                    to[i] = r < p.B && col < p.K ? __ldg((const uint4*)(p.x + (size_t)r * p.ldx + col)) : make_uint4(0u, 0u, 0u, 0u);
                }
                bits = p.act_bits && col < p.K ? __ldg(p.act_bits + (col >> 5)) >> (col & 31) : 0xFFu;
                if (col + 8 > p.K) bits &= (1u << max(p.K - col, 0)) - 1u;
            };
            fetch(k0, v[0], on[0]);
            if (nk > 1) fetch(k0 + 1, v[1], on[1]);
            int slot = 0;
            bool ok = true;
            for (int n = 0; n < nk && ok; n += 2) {
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const int last = n + j - p.sx;
                    if (n + j >= nk) break;
                    if (last >= 0 && !__all_sync(0xffffffffu, wait_or_abort(smem_u32(&x_empty[last % kRing]),
                                                                            (uint32_t)(last / kRing) & 1u, abort_flag,
                                                                            p.wait_limit))) {
                        if (lane == 0) flag_abort(abort_flag, p.status);
                        ok = false;
                        break;
                    }
                    unsigned char* dst = smem + (uint32_t)slot * p.x_bytes;
                    uint32_t m[4];
#pragma unroll
                    for (int e = 0; e < 4; e++)  // columns 2e, 2e+1 of the chunk
                        m[e] = ((on[j] >> (2 * e)) & 1u ? 0x0000FFFFu : 0u) | ((on[j] >> (2 * e + 1)) & 1u ? 0xFFFF0000u : 0u);
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        if (4 * i >= p.B && n + j >= p.sx) break;  // rows past the last stay zero
                        const int r = r0 + 4 * i;
                        uint32_t w[4] = {v[j][i].x, v[j][i].y, v[j][i].z, v[j][i].w};
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const uint32_t ge = (w[e] | 0x80008000u) - tb;  // bits 15 and 31: not below t
                            w[e] &= m[e] & prmt(ge, ge, 0xBB99u);
                        }
                        *(uint4*)(dst + 128 * r + ((c ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (n + j + 2 < nk) fetch(k0 + n + j + 2, v[j], on[j]);
                    if (++slot == p.sx) slot = 0;
                }
                if (!ok) break;
                fence_proxy_async_smem();  // generic stores -> tensor-core reads
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&x_full[n % kRing]));
                    if (n + 1 < nk) mbar_arrive(smem_u32(&x_full[(n + 1) % kRing]));
                }
            }
        } else if (lane == 0) {  // --------------------------------- token tiles
            for (int n = 0, slot = 0; n < nk; n++) {
                const int last = n - p.sx;
                if (last >= 0 && !wait_or_abort(smem_u32(&x_empty[last % kRing]), (uint32_t)(last / kRing) & 1u, abort_flag,
                                                p.wait_limit)) {
                    flag_abort(abort_flag, p.status);
                    break;
                }
                const uint32_t bar = smem_u32(&x_full[n % kRing]);
                const uint32_t dst = sbase + (uint32_t)slot * p.x_bytes;
                const int k = k0 + n;
                const bool second = MODE == kDx && k >= p.seg;
                mbar_arrive_expect_tx(bar, p.x_bytes);
                for (int h = 0; h < p.nh; h++)
                    tma_load_2d(dst + (uint32_t)(h * tok * 128), second ? &tx1 : &tx0, kBK * (second ? k - p.seg : k),
                                m0 + h * tok, bar);
                if (++slot == p.sx) slot = 0;
                x_issued++;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMAs
        const uint32_t idesc = idesc_f16(128, tok) | (MODE == kDx ? 1u << 15 : 0u);
        // the same operand bytes, 16 of the reduction a slice
        constexpr uint32_t kSliceA = MODE == kDx ? 256u : 4096u;
        const uint64_t ad0 = MODE == kDx ? umma_desc_plain(sbase + p.off_w, 128, 1024) : umma_desc_plain(sbase + p.off_w, 2048, 128);
        const uint64_t bd0 = umma_desc_sw128(sbase);
        uint32_t xo = 0, wo = 0;  // the slots' offsets
        for (int n = 0; n < nk; n++) {
            const uint32_t ph = (uint32_t)(n / kRing) & 1u;
            if (!__all_sync(0xffffffffu, wait_or_abort(smem_u32(&x_full[n % kRing]), ph, abort_flag, p.wait_limit) &&
                                             wait_or_abort(smem_u32(&w_full[n % kRing]), ph, abort_flag, p.wait_limit))) {
                if (lane == 0) flag_abort(abort_flag, p.status);
                break;
            }
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < kBK / 16; j++) {
                    const uint64_t ad = ad0 + ((wo + kSliceA * j) >> 4), bd = bd0 + ((xo + 32u * j) >> 4);
                    const uint32_t acc = tmem + (p.n_acc > 1 ? (uint32_t)(p.MT * j) : 0u);
                    const uint32_t add = n > 0 || (j > 0 && p.n_acc == 1) ? 1u : 0u;
                    umma_f16(acc, ad, bd, idesc, add);
                    if (p.nh > 1) umma_f16(acc + (uint32_t)tok, ad, bd + (uint32_t)(tok * 128 >> 4), idesc, add);
                }
                umma_commit(smem_u32(&x_empty[n % kRing]));
                umma_commit(smem_u32(&w_empty[n % kRing]));
            }
            __syncwarp();
            xo = xo + p.x_bytes == (uint32_t)p.sx * p.x_bytes ? 0u : xo + p.x_bytes;
            wo = wo + kWBytes == (uint32_t)p.sw * kWBytes ? 0u : wo + kWBytes;
        }
        if (elect_one()) {
            umma_commit(smem_u32(acc_full));
            umma_commit(smem_u32(drain));
        }
        __syncwarp();
        (void)mbar_drain(smem_u32(drain), 0);
        __syncwarp();
    } else if (warp == 2) {
        // ---------------------------------------------------------- compressed tiles
        // A lane for each tile of 16 steps; the two lanes of a step take their turn together.
        const int q = lane & 1;
        int slot = lane >> 1;
        while (slot >= p.sr) slot -= p.sr;
        for (int base = 0; base < nk; base += 16) {
            const int n = base + (lane >> 1), last = n - p.sr;
            const TileAt t = tile_at<MODE>(p, wt, k0 + n, q);
            const DirectLayer& L = p.L[t.w];
            // outside the section, or larger than the header allows: no values
            const bool in = n < nk && t.strip >= 0;
            const bool fits = in && u1 >= u0 && u1 <= L.values_units && 16u * (uint64_t)(u1 - u0) <= p.val_slot - 16u;
            if (in && !fits) raise_status(p.status, SPW_ERR_FORMAT);
            const uint32_t vbytes = fits ? 16u * (u1 - u0) : 0u;
            const uint64_t* bits = L.bitmaps + ((size_t)(in ? t.strip : 0) * p.n_ktiles + t.kt) * kTileCols;
            const uint16_t* vals = L.values + (size_t)u0 * 8;
            const uint32_t bar = smem_u32(&r_full[n % kRing]);
            const uint32_t dst = sbase + p.off_raw + (uint32_t)slot * p.raw_bytes;
            pointers(base + 16);
            bool ok = true;
            for (int j = 0; j < 16 && base + j < nk; j++) {
                // both lanes of a step issue, or none: what is in flight is then known
                const bool turn = lane >> 1 == j;
                ok = __all_sync(0xffffffffu, !turn || last < 0 ||
                                                 wait_or_abort(smem_u32(&r_empty[last % kRing]), (uint32_t)(last / kRing) & 1u,
                                                               abort_flag, p.wait_limit));
                if (!ok) {
                    if (lane == 0) flag_abort(abort_flag, p.status);
                    break;
                }
                if (turn) {
                    r_info[2 * (n % kRing) + q] = fits ? vbytes >> 4 : 0xFFFFFFFFu;
                    mbar_arrive_expect_tx(bar, fits ? 512u + vbytes : 0u);
                    if (fits) bulk_g2s(dst + 512u * q, bits, 512u, bar);
                    if (vbytes) bulk_g2s(dst + 1024u + p.val_slot * q, vals, vbytes, bar);
                }
                __syncwarp();
                r_issued++;
            }
            if (!ok) break;
            slot += 16;
            while (slot >= p.sr) slot -= p.sr;
        }
    } else {
        // ---------------------------------------------------------- decoders
        // Group g takes the steps g, g + GROUPS, ...; its warp takes columns 32 half .. of tile q.
        // Lane l owns rows 2l and 2l+1: bits b and b+1 of one half of each column's word.
        const int d = warp - kFirstDecoder, q = (d >> 1) & 1, half = d & 1;
        unsigned char* rec = smem + p.off_rec + kRecBytes * d;
        const int up = 30 - 2 * (lane & 15);
        const uint32_t above = 0xFFFFFFFEu << (2 * (lane & 15));
        const uint4* recp = (const uint4*)(rec + (lane < 16 ? 0 : 272));
        // dense tiles: kEp, kFfn [8 columns][16 row groups]; kDx [8 columns of each tile][8 row groups]
        const uint32_t step = MODE == kDx ? 1024u : 2048u;
        const uint32_t mine = (MODE == kDx ? 8192u : 1024u) * q + 4u * step * half + 32u * lane;
        const uint32_t swap = ((uint32_t)lane >> 2) & 1u;  // the 8 lanes of a store in distinct banks
        int rslot = d >> 2, wslot = d >> 2;
        while (rslot >= p.sr) rslot -= p.sr;
        while (wslot >= p.sw) wslot -= p.sw;
        for (int n = d >> 2; n < nk; n += GROUPS) {
            const uint32_t ph = (uint32_t)(n / kRing) & 1u;
            if (!__all_sync(0xffffffffu, wait_or_abort(smem_u32(&r_full[n % kRing]), ph, abort_flag, p.wait_limit))) {
                if (lane == 0) flag_abort(abort_flag, p.status);
                break;
            }
            const uint32_t units = r_info[2 * (n % kRing) + q];
            bool good = units != 0xFFFFFFFFu;
            if (good) {
                const unsigned char* raw = smem + p.off_raw + (uint32_t)rslot * p.raw_bytes;
                const uint4 bw = *(const uint4*)(raw + 512 * q + 16 * lane);  // columns 2l, 2l+1
                const int cl0 = __popc(bw.x), c0 = cl0 + __popc(bw.y);
                const int cl1 = __popc(bw.z), c1 = cl1 + __popc(bw.w);
                const int incl = warp_inclusive_scan(c0 + c1, lane);
                const int total = __shfl_sync(0xffffffffu, incl, 31);
                // bitmaps and pointers that disagree: reported, and the tile counts as empty
                good = (uint32_t)(total + 7) / 8u == units;
                if (!good && half == 0 && lane == 0) raise_status(p.status, SPW_ERR_FORMAT);
                if (good && (lane >> 4) == half) {
                    const uint32_t a0 = smem_u32(raw) + 1024u + p.val_slot * q + 2u * (uint32_t)(incl - c0 - c1);
                    const uint32_t a1 = a0 + 2u * (uint32_t)c0;
                    uint4* to = (uint4*)(rec + 16 * (lane & 15));
                    to[0] = make_uint4(bw.x, a0 + 2u * (uint32_t)cl0, bw.z, a1 + 2u * (uint32_t)cl1);
                    to[17] = make_uint4(bw.y, a1, bw.w, a1 + 2u * (uint32_t)c1);
                }
            }
            __syncwarp();
            const int last = n - p.sw;
            if (last >= 0 && !__all_sync(0xffffffffu, wait_or_abort(smem_u32(&w_empty[last % kRing]), (uint32_t)(last / kRing) & 1u,
                                                                    abort_flag, p.wait_limit))) {
                if (lane == 0) flag_abort(abort_flag, p.status);
                break;
            }
            unsigned char* out = smem + p.off_w + (uint32_t)wslot * kWBytes + mine;
#pragma unroll
            for (int g = 0; g < 4; g++) {
                uint32_t o0[4] = {0u, 0u, 0u, 0u}, o1[4] = {0u, 0u, 0u, 0u};
                if (good) {
#pragma unroll
                    for (int pr = 0; pr < 4; pr++) decode_pair(recp[4 * g + pr], above, up, o0[pr], o1[pr]);
                }
                const uint4 s0 = make_uint4(o0[0], o0[1], o0[2], o0[3]), s1 = make_uint4(o1[0], o1[1], o1[2], o1[3]);
                *(uint4*)(out + g * step + 16u * swap) = swap ? s1 : s0;
                *(uint4*)(out + g * step + 16u * (1u - swap)) = swap ? s0 : s1;
            }
            fence_proxy_async_smem();  // generic stores -> tensor-core reads
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&w_full[n % kRing]));
                mbar_arrive(smem_u32(&r_empty[n % kRing]));
            }
            rslot += GROUPS;
            while (rslot >= p.sr) rslot -= p.sr;
            wslot += GROUPS;
            while (wslot >= p.sw) wslot -= p.sw;
        }
        if (!__all_sync(0xffffffffu, wait_or_abort(smem_u32(acc_full), 0, abort_flag, p.wait_limit)) && lane == 0)
            flag_abort(abort_flag, p.status);
        tc_fence_after();
    }
    __syncthreads();

    // ---------------------------------------------------------------- result
    // p.chunk tokens at a time: every CTA of the cluster puts its piece into its shared memory
    // ([token][128 rows], over the slots, which are no longer in use), then adds the pieces of its
    // share of the tokens and writes them.  (After an abort the values mean nothing.)
    float* buf = (float*)smem;
    for (int c0 = 0; c0 < p.MT; c0 += p.chunk) {
        const int n = min(p.chunk, p.MT - c0);
        if (warp >= kFirstDecoder) {
            const int d = warp - kFirstDecoder, quarter = warp & 3;
            for (int c = 32 * (d >> 2); c < n; c += 32 * GROUPS) {
                uint32_t r[32];
                tmem_ld32(tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)(c0 + c), r);
                for (int a = 1; a < p.n_acc; a++) {
                    uint32_t r2[32];
                    tmem_ld32(tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)(a * p.MT + c0 + c), r2);
#pragma unroll
                    for (int j = 0; j < 32; j++) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(r2[j]));
                }
#pragma unroll
                for (int j = 0; j < 32; j++)
                    if (c + j < n) buf[(c + j) * 128 + 32 * quarter + lane] = __uint_as_float(r[j]);
            }
        }
        __syncwarp();
        if (p.parts > 1) cluster_sync_all();
        else __syncthreads();
        const int t0 = part * n / p.parts, t1 = (part + 1) * n / p.parts;
        constexpr int kLanes = MODE == kFfn ? 16 : 32;  // lanes of a token's row
        for (int i = threadIdx.x; i < (t1 - t0) * kLanes; i += kThreads) {
            const int t = t0 + i / kLanes, r = 4 * (i % kLanes);
            const int m = m0 + c0 + t;
            if (m >= p.o.rows) break;
            auto sum = [&](int row, float (&v)[4]) {
                const uint32_t at = smem_u32(buf + t * 128 + row);
                v[0] = v[1] = v[2] = v[3] = 0.0f;
                for (int z = 0; z < p.parts; z++) {
                    const float4 f = p.parts > 1 ? ld_cluster_f4(map_to_rank(at, (uint32_t)z)) : *(const float4*)(buf + t * 128 + row);
                    v[0] += f.x;
                    v[1] += f.y;
                    v[2] += f.z;
                    v[3] += f.w;
                }
            };
            float v[4];
            sum(r, v);
            if constexpr (MODE == kFfn) {
                const int col = 64 * wt + r;
                float u[4];
                sum(64 + r, u);
                if (col < p.o.cols) {
                    if (p.o.G) {
                        store4(p.o.G + (size_t)m * p.o.ldg, col, p.o.cols, p.o.vec & 4, v);
                        store4(p.o.U + (size_t)m * p.o.ldu, col, p.o.cols, p.o.vec & 8, u);
                    }
                    act_all(v, p.o.act);
#pragma unroll
                    for (int e = 0; e < 4; e++) v[e] *= u[e];
                    store4(p.o.Y + (size_t)m * p.o.ldy, col, p.o.cols, p.o.vec & 1, v);
                }
            } else {
                const int col = 128 * wt + r;
                if (col < p.o.cols) {
                    if constexpr (MODE == kEp || MODE == kDecode) {
                        if (p.o.bias) add4(p.o.bias, col, p.o.cols, true, v);
                        act_all(v, p.o.act);
                        if (p.o.residual) add4(p.o.residual + (size_t)m * p.o.ldr, col, p.o.cols, p.o.vec & 2, v);
                    }
                    store4(p.o.Y + (size_t)m * p.o.ldy, col, p.o.cols, p.o.vec & 1, v);
                }
            }
        }
        // before the next chunk overwrites it, or this CTA leaves: no piece is being read
        __syncwarp();
        if (p.parts > 1) cluster_sync_all();
        else __syncthreads();
    }
    if (*abort_flag) {  // the copies this CTA armed: for each barrier the phase of its last use
        if (warp == 0 && lane == 0)
            for (int i = x_issued > kRing ? x_issued - kRing : 0; i < x_issued; i++)
                (void)mbar_drain(smem_u32(&x_full[i % kRing]), (uint32_t)(i / kRing) & 1u);
        if (warp == 2 && lane == 0)
            for (int i = r_issued > kRing ? r_issued - kRing : 0; i < r_issued; i++)
                (void)mbar_drain(smem_u32(&r_full[i % kRing]), (uint32_t)(i / kRing) & 1u);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.tmem_cols) : "memory");
    }
}

// ------------------------------------------------------------------ host side
struct DirectPlan {
    int groups, parts, wt, m_tiles, MT, nh, n_acc, steps, sx, sw, sr, chunk;
    uint32_t x_bytes, val_slot, raw_bytes, tmem_cols, off_w, off_raw, off_rec, off_bar;
    size_t smem;
    double cost;
};

constexpr uint32_t kBarBytes = 8u * (6 * kRing + 2) + 8u * kRing + 16u;

// Slots for a CTA with `limit` bytes of shared memory.
bool fit(DirectPlan* g, uint32_t limit) {
    static const int opt[][3] = {{4, 4, 8}, {4, 4, 6}, {4, 4, 5}, {3, 4, 5}, {3, 4, 4}, {2, 4, 4}, {2, 3, 4}, {2, 3, 3}, {2, 2, 3}, {2, 2, 2}};
    for (const int* o : opt) {
        if (g->groups == 2 && o[1] > 3) continue;
        g->sx = o[0];
        g->sw = o[1];
        g->sr = o[2];
        g->off_w = (uint32_t)g->sx * g->x_bytes;
        g->off_raw = g->off_w + (uint32_t)g->sw * kWBytes;
        g->off_rec = g->off_raw + (uint32_t)g->sr * g->raw_bytes;
        g->off_bar = g->off_rec + kRecBytes * 4u * (uint32_t)g->groups;
        g->chunk = (int)(g->off_rec / 512u) / 32 * 32;  // over the slots
        if (g->chunk > g->MT) g->chunk = g->MT;
        if (g->chunk < 16) continue;
        g->smem = (size_t)g->off_bar + kBarBytes + 1024;
        if (g->smem <= limit) return true;
    }
    return false;
}

template <int MODE, int GROUPS>
const void* kernel_of() { return (const void*)direct_kernel<MODE, GROUPS>; }
const void* kernel_for(int mode, int groups) {
    switch (mode) {
        case kEp: return groups == 2 ? kernel_of<kEp, 2>() : kernel_of<kEp, 4>();
        case kFfn: return groups == 2 ? kernel_of<kFfn, 2>() : kernel_of<kFfn, 4>();
        case kDx: return groups == 2 ? kernel_of<kDx, 2>() : kernel_of<kDx, 4>();
        default: return groups == 2 ? kernel_of<kDecode, 2>() : kernel_of<kDecode, 4>();
    }
}

// CTAs in clusters of `parts` that are resident at one CTA an SM (with the largest shared memory
// of the variant), per device; 0 when the query fails.
int resident(int groups, int parts) {
    static int cache[kMaxDevices][2][kMaxParts + 1];
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    std::lock_guard<std::mutex> lock(mu);
    int& n = cache[dev][groups == 2][parts];
    if (!n) {
        const int smem = groups == 2 ? kSmemLimit / 2 - 1024 : kSmemLimit;
        for (int mode : {kEp, kFfn, kDx, kDecode})
            if (cudaFuncSetAttribute(kernel_for(mode, groups), cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
                (void)cudaGetLastError();
                return 0;
            }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)parts);
        cfg.blockDim = dim3((unsigned)threads_of(groups));
        cfg.dynamicSmemBytes = (size_t)smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)parts;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int c = 0;
        if (cudaOccupancyMaxActiveClusters(&c, kernel_for(kEp, groups), &cfg) != cudaSuccess) c = 0;
        (void)cudaGetLastError();
        n = c * parts;
    }
    return n;
}

int search_plan(int mode, const spw_format* h, const spw_format* h2, int M, uint32_t units, DirectPlan* best) {
    best->cost = -1.0;
    if (M > kMaxDim || h->N > kMaxDim || h->K > kMaxDim) return SPW_ERR_UNSUPPORTED;
    for (int groups = 2; groups <= 4; groups += 2)
        for (int cap = kMaxTok; cap >= 64; cap /= 2) {
            DirectPlan g;
            memset(&g, 0, sizeof(g));
            g.groups = groups;
            g.wt = mode == kEp ? (int)((h->N + 127) / 128) : mode == kFfn ? (int)h->n_strips : (int)((h->n_ktiles + 1) / 2);
            g.steps = mode == kDx ? (int)h->n_strips * (h2 ? 2 : 1) : (int)h->n_ktiles;
            g.m_tiles = (int)(((long long)M + cap - 1) / cap);
            const int per = (int)(((long long)M + g.m_tiles - 1) / g.m_tiles);
            g.nh = per > 256 ? 2 : 1;
            g.MT = (int)round_up_u64((uint64_t)per, 16u * (unsigned)g.nh);
            g.x_bytes = (uint32_t)g.MT * 128u;  // a multiple of 1024: the swizzle's alignment
            g.val_slot = (uint32_t)round_up_u64(16ull * units + 16, 16);
            g.raw_bytes = (uint32_t)round_up_u64(1024u + 2u * g.val_slot, 128);
            g.n_acc = g.MT <= 64 ? 4 : 1;
            g.tmem_cols = 32;  // 32 columns are read at a time
            while (g.tmem_cols < (uint32_t)((g.n_acc - 1) * g.MT) + round_up_u64((uint64_t)g.MT, 32)) g.tmem_cols <<= 1;
            if (groups == 2 && g.tmem_cols > 256) continue;  // two CTAs share an SM's 512 columns
            if (!fit(&g, groups == 2 ? kSmemLimit / 2 - 1024 : kSmemLimit)) continue;
            const long long tiles = (long long)g.wt * g.m_tiles;
            if (tiles * kMaxParts > 0x3fffffffll) continue;
            for (int parts = 1; parts <= kMaxParts && parts <= g.steps; parts++) {
                const int slots = resident(groups, parts);
                if (slots <= 0) continue;
                const double steps = (double)((g.steps + parts - 1) / parts);
                // Fitted to measured times of every split (9 weights, 16 to 400 tokens; the plan it
                // picks is within 0.1 % of the fastest on average): a step of two tiles (decoding, and
                // shared memory's share of the tokens; above 256 tokens all SMs' token tiles come near
                // what L2 delivers), and what a CTA takes before the first and after the last, most of
                // it the exchange of the pieces.  (4096 x 4096, 4 pieces of 16 steps: 16.2 us at 16
                // tokens, 19.2 at 128, 23.0 at 256, 32.4 at 512.)  CTAs of two groups go two to an SM,
                // where the one works while the other starts or ends but both decode more slowly:
                // better where whole waves fit badly (11008 x 4096 at 16 tokens 34 us against 39, gated
                // 67 against 74; 4096 x 4096 18.8 against 16.4).
                const double ends = 5.6 + (parts > 1 ? 0.9 : 0.0) + 0.0235 * g.MT;
                double cost;
                if (groups == 4) {
                    const double step = 0.55 + 0.0005 * g.MT + (g.MT > 256 ? 0.00055 * (g.MT - 256) : 0.0);
                    cost = (double)((tiles * parts + slots - 1) / slots) * (steps * step + ends);
                } else {
                    const long long full = tiles * parts / (2 * slots), rest = tiles * parts % (2 * slots);
                    const double shared = steps * (1.1 + 0.004 * g.MT) + ends, alone = steps * (0.7 + 0.002 * g.MT) + ends;
                    cost = (double)full * shared + (rest == 0 ? 0.0 : rest <= slots ? alone : shared);
                }
                if (best->cost < 0 || cost < best->cost * 0.98) {
                    *best = g;
                    best->parts = parts;
                    best->cost = cost;
                }
            }
        }
    return best->cost < 0 ? SPW_ERR_UNSUPPORTED : SPW_OK;
}

// A call asks for its plan up to three times (workspace, choice, launch): the thread's last
// plans are kept by what they follow from.
int plan_direct(int mode, const spw_format* h, const spw_format* h2, int M, DirectPlan* out) {
    struct Key {
        int dev, mode, weights, M;
        uint32_t N, K, units;
    };
    struct Entry {
        Key key;
        DirectPlan plan;
        int rc;
        bool used;
    };
    static thread_local Entry cache[4];
    static thread_local unsigned turn;
    Key key;
    memset(&key, 0, sizeof(key));
    if (cudaGetDevice(&key.dev) != cudaSuccess) return SPW_ERR_CUDA;
    key.mode = mode;  // (kDecode plans as kEp)
    key.weights = h2 ? 2 : 1;
    key.M = M;
    key.N = h->N;
    key.K = h->K;
    key.units = h2 && h2->max_tile_units > h->max_tile_units ? h2->max_tile_units : h->max_tile_units;
    for (Entry& e : cache)
        if (e.used && memcmp(&e.key, &key, sizeof(key)) == 0) {
            *out = e.plan;
            return e.rc;
        }
    Entry& e = cache[turn++ % 4];
    e.key = key;
    e.rc = search_plan(mode, h, h2, M, key.units, &e.plan);
    e.used = true;
    *out = e.plan;
    return e.rc;
}

}  // namespace

double direct_cost(int mode, const spw_format* h, const spw_format* h2, int M) {
    DirectPlan g;
    return plan_direct(mode, h, h2, M, &g) == SPW_OK ? g.cost : -1.0;
}

int direct_launch(const DirectCall& c, cudaStream_t s) {
    DirectPlan g;
    int rc = plan_direct(c.mode == kDecode ? (int)kEp : c.mode, c.h[0], c.h[1], c.M, &g);
    if (rc != SPW_OK) return rc;
    DirectParams p;
    memset(&p, 0, sizeof(p));
    CUtensorMap tx[2];
    for (int w = 0; w < 2; w++) {
        const spw_format* h = c.h[w];
        if (h) {
            const uint8_t* buf = (const uint8_t*)c.buf[w];
            p.L[w].bitmaps = (const uint64_t*)(buf + h->off_bitmaps);
            p.L[w].tileptr = (const uint32_t*)(buf + h->off_tileptr);
            p.L[w].values = (const uint16_t*)(buf + h->off_values);
            p.L[w].values_units = (h->bytes_total - h->off_values) / 16;
        }
        if (c.mode == kDecode) {
            memset(&tx[w], 0, sizeof(tx[w]));  // not read
        } else if (c.x[w]) {
            rc = encode_map_f16(&tx[w], c.x[w], c.mode == kDx ? c.h[0]->N : c.h[0]->K, (uint64_t)c.M, c.ldx_bytes[w], kBK,
                                (uint32_t)(g.MT / g.nh));
            if (rc != SPW_OK) return rc;
        } else {
            tx[w] = tx[0];
        }
    }
    p.o = c.out;
    p.n_strips = (int)c.h[0]->n_strips;
    p.n_ktiles = (int)c.h[0]->n_ktiles;
    p.steps = g.steps;
    p.seg = (int)c.h[0]->n_strips;
    p.parts = g.parts;
    p.m_tiles = g.m_tiles;
    p.MT = g.MT;
    p.nh = g.nh;
    p.n_acc = g.n_acc;
    p.sx = g.sx;
    p.sw = g.sw;
    p.sr = g.sr;
    p.chunk = g.chunk;
    p.x_bytes = g.x_bytes;
    p.val_slot = g.val_slot;
    p.raw_bytes = g.raw_bytes;
    p.tmem_cols = g.tmem_cols;
    p.off_w = g.off_w;
    p.off_raw = g.off_raw;
    p.off_rec = g.off_rec;
    p.off_bar = g.off_bar;
    p.status = device_status_ptr();
    p.wait_limit = wait_limit_cycles();
    if (!p.status) return SPW_ERR_CUDA;
    p.x = c.x[0];
    p.act_bits = c.act_bits;
    p.B = c.M;
    p.K = (int)c.h[0]->K;
    p.ldx = c.ldx;
    p.t_bits = 1;
    if (c.mode == kDecode && c.t > 0.0f) {
        // round up: the nearest fp16, or the next one (the bits of positive fp16 count upward)
        const __half h = __float2half_rn(c.t);
        uint16_t bits;
        memcpy(&bits, &h, 2);
        if (__half2float(h) < c.t) bits++;
        p.t_bits = bits < 1 ? 1 : bits;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)g.wt * g.m_tiles * g.parts));
    cfg.blockDim = dim3((unsigned)threads_of(g.groups));
    cfg.dynamicSmemBytes = g.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)g.parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = c.early ? 2 : 1;
    void* args[3] = {&tx[0], &tx[1], &p};
    SPW_CUDA_TRY(cudaLaunchKernelExC(&cfg, kernel_for(c.mode, g.groups), args));
    return SPW_OK;
}

}  // namespace spw
