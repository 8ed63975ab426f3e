// Shared by the tensor-core kernels of the gated delta rule: the per-chunk
// operand block that the chunk-parallel kernel writes and the chains read.
#pragma once

#include "gdr_internal.cuh"
#include "inter_common.cuh"
#include "tc_common.cuh"

namespace mdn {
namespace gdr {

// With la the decay sums inside a chunk and L_{r,i} = exp(la_r - la_i),
//     A_{r,i}   = L_{r,i} beta_i k_r.k_i          (i < r),  T = (I + A)^{-1},
//     Att_{r,i} = scale L_{r,i} beta_i q_r.k_i    (i <= r),
// the chunk form of the rule is, with S the state entering the chunk,
//     Y = V - Diag(D) K S,  Vtilde = T Y,  o = scale Diag(D) Q S + Att Vtilde,
//     S' = aC S + K^T Diag(gam) Vtilde,
// D_r = exp(la_r), gam_i = beta_i exp(la_C - la_i), aC = exp(la_C).
//
// One block per chunk and head: bf16 images of 64 rows x 128 bytes with the
// 128-byte swizzle (K-major operands), T in two terms T = T_hi + T_lo (16 bits
// of significand together), then the fp32 record.
constexpr uint32_t kBlkThi = 0;
constexpr uint32_t kBlkAtt = 8192;    // directly behind T_hi: one M = 128 operand [T_hi; Att]
constexpr uint32_t kBlkTlo = 16384;
constexpr uint32_t kBlkImg = 24576;   // bytes of the images
constexpr uint32_t kBlkRec = 24576;   // 256 floats
constexpr uint32_t kBlkBytes = 25600;
// record
constexpr int kRecD = 0;      // D_r
constexpr int kRecDq = 64;    // scale D_r
constexpr int kRecGam = 128;  // gam_r
constexpr int kRecB = 192;    // [192]: aC
constexpr int kRecFloats = 256;

// x as two bf16 terms, eight values: 16 bytes each.
__device__ __forceinline__ void split8(const float* x, uint4& hi, uint4& lo)
{
    float h[8], l[8];
    hi = tc::bf16x8(x);
    tc::unpack_bf16x8(hi, h);
#pragma unroll
    for (int e = 0; e < 8; ++e) l[e] = x[e] - h[e];
    lo = tc::bf16x8(l);
}

// Two values as two bf16 terms each.
__device__ __forceinline__ void unpack2(uint32_t w, float& x0, float& x1)
{
    x0 = __uint_as_float(w << 16);
    x1 = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo)
{
    float h0, h1;
    hi = tc::pack_bf16(x0, x1);
    unpack2(hi, h0, h1);
    lo = tc::pack_bf16(x0 - h0, x1 - h1);
}

// 16 lanes x 8 N columns of TMEM (lanes 32 (warp % 4) .. + 15): thread t holds, of
// each 8-column piece, columns 2 (t % 4), + 1 of row t / 4 in v[4 i], v[4 i + 1] and of
// row t / 4 + 8 in v[4 i + 2], v[4 i + 3].  Warp-collective.
template <int N>
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, float* v)
{
    if constexpr (N == 1) {
        uint32_t r[4];
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(taddr));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
    } else if constexpr (N == 2) {
        uint32_t r[8];
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) tmem_ld_16x256<2>(taddr + 8 * i, v + 4 * i);
    }
}

// D[tmem] (+)= A B and its commit, issued by one elected lane of a converged warp: the
// operands stay in uniform registers, and an instruction is issued every 32 cycles
// instead of the 54 it takes from inside a one-lane branch.
__device__ __forceinline__ void mma_bf16_elect(uint32_t d, uint64_t adesc, uint64_t bdesc,
                                               uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_commit_elect(uint64_t* bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(
            sm100::smem_u32(bar))
        : "memory");
}

// TMA map over [rows..., heads, D] bf16; box = {box_d, 1, box_rows, 1}.  Batches keep
// their own dimension so that rows past T read as zeros.
bool make_rows_map(CUtensorMap* map, const void* base, const Args& a, int heads, int box_d,
                   CUtensorMapSwizzle swizzle, int box_rows = kChunk);

// The operand blocks of every chunk and head (a.blk).
cudaError_t launch_operands_tc(const Args& a, cudaStream_t s);

}  // namespace gdr
}  // namespace mdn
