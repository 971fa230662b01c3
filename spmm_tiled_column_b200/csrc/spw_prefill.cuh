// spw_prefill.cuh -- what the two forms of the prefill products with an epilogue share
// (spmm_direct.cu for few tokens, gemm.cu for many): the kinds of product, and the results
// and operands of their epilogues.
#pragma once

#include "spw_act.cuh"
#include "spw_internal.cuh"

namespace spw {

// kEp: act(X W^T + bias) + residual.  kFfn: act(X Wg^T) * (X Wu^T).  kDx: sum of dY W over one
// or two weights.  kDv: dY^T X at the kept positions (gemm.cu only).  kDecode: kEp for at most
// 16 rows with the decode's rule (spmm_direct.cu only).
enum Mode { kEp, kFfn, kDx, kDv, kDecode };

struct PrefillOut {
    uint16_t* Y;
    const uint16_t* bias;
    const uint16_t* residual;
    uint16_t* G;
    uint16_t* U;
    int ldy, ldr, ldg, ldu, act;
    int vec;         // bit 0: Y, 1: residual, 2: G, 3: U take 16-byte accesses;
                     // 4: Y and residual, 5: G, 6: U take 4-byte ones
    int rows, cols;  // of the result (kFfn: of H)
};

// Largest M, N and K of these products: rows and columns are numbered in int up to the end of the
// last tile (at most 512 past the last row).
constexpr long long kMaxDim = 0x7ffff000;

// A product by the direct form: the weights (h2 null for one), the activations of each
// segment (kDx: dY of each weight; else one), their row strides in bytes.
struct DirectCall {
    int mode;
    const spw_format* h[2];
    const void* buf[2];
    const uint16_t* x[2];
    uint64_t ldx_bytes[2];
    int M;
    PrefillOut out;
    // kDecode: the rows' stride in elements, the threshold and the column set (or null)
    int ldx;
    float t;
    const uint32_t* act_bits;
    bool early;  // may start while the kernel before it, of the same call, still runs
};

// Estimated time in microseconds (< 0: the form cannot run this product), and the launch.
double direct_cost(int mode, const spw_format* h, const spw_format* h2, int M);
// PrefillOut::vec from its leading dimensions (every pointer is 16-byte aligned).
int vec_bits(const PrefillOut& o);
int direct_launch(const DirectCall& c, cudaStream_t s);

// Shared-memory loads of 16 bits, zero-extended (not volatile: see lds_u16).
__device__ inline uint32_t lds_u16_at(uint32_t addr) {
    uint32_t v;
    asm("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ inline uint32_t lds_u16_before(uint32_t addr) {
    uint32_t v;
    asm("ld.shared.u16 %0, [%1+-2];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ inline uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

// Two neighbouring columns of a compressed tile, rows r and r + 1 (r even) of one 32-row half:
// rec = {bits, end, bits, end} of the columns' halves, end the shared-memory address behind
// the half's last kept value; above = the bits of rows r + 1 and up, up = 30 - r.  The kept
// rows from r + 1 upward are the last popc of that half, so row r + 1's value stands at end -
// 2 popc and row r's just before it (what is loaded for a dropped row belongs to another row
// or to the slack around the values).  A column's two bits are shifted to bit 31, whose sign
// prmt spreads over the column's 16 bits as the mask: 21 instructions for four entries,
// where tests and selects took twice as many.
__device__ inline void decode_pair(const uint4& rec, uint32_t above, int up, uint32_t& row0, uint32_t& row1) {
    uint32_t a, b;
    asm("mad.lo.s32 %0, %1, -2, %2;" : "=r"(a) : "r"(__popc(rec.x & above)), "r"(rec.y));
    asm("mad.lo.s32 %0, %1, -2, %2;" : "=r"(b) : "r"(__popc(rec.z & above)), "r"(rec.w));
    const uint32_t ta = rec.x << up, tb = rec.z << up;
    row1 = prmt(lds_u16_at(a), lds_u16_at(b), 0x5410u) & prmt(ta, tb, 0xFFBBu);
    row0 = prmt(lds_u16_before(a), lds_u16_before(b), 0x5410u) & prmt(ta << 1, tb << 1, 0xFFBBu);
}

}  // namespace spw
