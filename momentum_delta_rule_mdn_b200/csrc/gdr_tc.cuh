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

// TMA map over [rows..., heads, D] bf16; box = {box_d, 1, 64, 1}.  Batches keep
// their own dimension so that rows past T read as zeros.
bool make_rows_map(CUtensorMap* map, const void* base, const Args& a, int heads, int box_d,
                   CUtensorMapSwizzle swizzle);

// The operand blocks of every chunk and head (a.blk).
cudaError_t launch_operands_tc(const Args& a, cudaStream_t s);

}  // namespace gdr
}  // namespace mdn
