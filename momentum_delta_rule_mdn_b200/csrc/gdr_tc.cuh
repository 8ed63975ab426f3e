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

// The backward pass's block.  Its chain carries E = dv / beta (finite where beta = 0,
// and dbeta = vtilde . E): with A'_{r,i} = beta_r L_{r,i} k_r.k_i (the row's beta) and
// Att'_{r,i} = scale L_{r,i} q_r.k_i,
//     E = T'^T (Att'^T dO + Diag(gamU) K G),   T' = (I + A')^{-1},   dv = beta E,
//     G <- aC G + Q^T Diag(Dq) dO - K^T Diag(D) dv,   gamU_i = exp(la_C - la_i).
// Everything here leads to fp32 gradients (of the gates and the entering state), so
// Att' is kept in two bf16 terms too.
constexpr uint32_t kBwdAttLo = 24576;
constexpr uint32_t kBwdImg = 32768;
constexpr uint32_t kBwdRecBytes = 1792;
constexpr uint32_t kBwdBytes = kBwdImg + kBwdRecBytes;
constexpr int kRecGamU = 192;  // exp(la_C - la_r)
constexpr int kRecBeta = 256;  // beta_r
constexpr int kRecBwdB = 320;  // [320]: aC

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

// x + y exactly, as a float and its rounding error (Knuth's two-sum)
__device__ __forceinline__ float two_sum(float x, float y, float& err)
{
    const float s = __fadd_rn(x, y), z = __fsub_rn(s, x);
    err = __fadd_rn(__fsub_rn(x, __fsub_rn(s, z)), __fsub_rn(y, z));
    return s;
}

// Gate vectors of a chunk: four vectors of 64 floats, vector v's 4-element piece g at
// base + (16 v + g) * stride.  p = block sum up to the token (two floats), beta, and
// beta_i exp(sum behind the token to the end of its block).
struct GateVec {
    uint8_t* base;
    uint32_t stride;
    __device__ __forceinline__ float4 get4(int v, int g) const {
        return *reinterpret_cast<const float4*>(base + (16 * v + g) * stride);
    }
    __device__ __forceinline__ float& at(int v, int i) const {
        return *reinterpret_cast<float*>(base + (16 * v + (i >> 2)) * stride + (i & 3) * 4);
    }
};
enum { kP = 0, kPlo = 1, kBeta = 2, kSbeta = 3 };

// One warp: the gate vectors, the block factors and the record of a chunk from
// its gates (tokens 2 lane, 2 lane + 1).
// (BWD: the backward block's record, and kSbeta without beta_i.)
template <bool BWD>
__device__ __forceinline__ void scan_gates(const GateVec& gv, float* btot, float* rec, float scale,
                                           const float (&ga)[2], const float (&gb)[2], int lane)
{
    const float a0 = ga[0] < -1e4f ? -1e4f : ga[0], a1 = ga[1] < -1e4f ? -1e4f : ga[1];
    float s1lo, hi, lo;
    const float s1 = two_sum(a0, a1, s1lo);
    hi = s1;
    lo = s1lo;
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
        const float h2 = __shfl_up_sync(0xffffffffu, hi, off, 8), l2 = __shfl_up_sync(0xffffffffu, lo, off, 8);
        if ((lane & 7) >= off) {
            float e;
            hi = two_sum(hi, h2, e);
            lo += l2 + e;
        }
    }
    float bh = __shfl_up_sync(0xffffffffu, hi, 1, 8), bl = __shfl_up_sync(0xffffffffu, lo, 1, 8);
    if ((lane & 7) == 0) bh = bl = 0.f;
    const float th = __shfl_sync(0xffffffffu, hi, 7, 8), tl = __shfl_sync(0xffffffffu, lo, 7, 8);
    float p[2], plo[2], e0;
    p[0] = two_sum(bh, a0, e0);
    plo[0] = bl + e0;
    p[1] = hi;
    plo[1] = lo;
    const int B = lane >> 3;
    float pre = 0.f, post = 0.f, all = 0.f;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const float t = __shfl_sync(0xffffffffu, th, 8 * b);
        if (b < B) pre += t;
        if (b > B) post += t;
        all += t;
    }
    const float fpre = expf(pre), fpost = expf(post);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = 2 * lane + e;
        const float ep = expf(p[e]), D_ = fpre * fmaf(ep, plo[e], ep);
        const float sx = expf((th - p[e]) + (tl - plo[e])), sb = gb[e] * sx;
        gv.at(kP, r) = p[e];
        gv.at(kPlo, r) = plo[e];
        gv.at(kBeta, r) = gb[e];
        gv.at(kSbeta, r) = BWD ? sx : sb;
        if (!rec) continue;
        rec[kRecD + r] = D_;
        rec[kRecDq + r] = scale * D_;
        rec[kRecGam + r] = sb * fpost;
        if (BWD) {
            rec[kRecGamU + r] = sx * fpost;
            rec[kRecBeta + r] = gb[e];
        }
    }
    if ((lane & 7) == 0) btot[B] = expf(th);
    if (lane == 0 && rec) rec[BWD ? kRecBwdB : kRecB] = expf(all);
}

// TMA map over [rows..., heads, D] bf16; box = {box_d, 1, box_rows, 1}.  Batches keep
// their own dimension so that rows past T read as zeros.
bool make_rows_map(CUtensorMap* map, const void* base, const Args& a, int heads, int box_d,
                   CUtensorMapSwizzle swizzle, int box_rows = kChunk);

// The same over [chunks * H] d x d matrices; box = {box_d, d, 1}.
bool make_states_map(CUtensorMap* map, const void* base, const Args& a, int box_d, CUtensorMapSwizzle swizzle);

// The operand blocks of every chunk and head (a.blk), each flagged in a.ready once it is
// written.  CTAs on SMs 0 .. reserve - 1 stop after `limit` chunks, so that a kernel launched
// as this one's programmatic dependent finds those SMs free early.
cudaError_t launch_operands_tc(const Args& a, cudaStream_t s, bool bwd, int reserve, int limit);

}  // namespace gdr
}  // namespace mdn
