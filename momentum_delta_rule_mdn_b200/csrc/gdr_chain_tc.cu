// The forward chain of the gated delta rule on sm_100a (formulas in gdr_tc.cuh):
// one CTA per chain and NS of its d_v columns, walking the chunks in order with
// the state in fp32 registers.
//
// Per chunk, three dependent rounds on the tensor cores and two products beside
// them (K^T is the K tile read MN-major; every right operand is MN-major):
//   A1 = K [S_hi | S_lo]                 (M 64, N 2 NS, K d)
//   Y  = V - Diag(D) K (S_hi + S_lo)     in fp32, as two bf16 terms
//   AT = T_hi [Y_hi | Y_lo] + T_lo [Y_hi | Y_lo]    (M 64, N 2 NS, K 64)
//   Vtilde = AT_hi + AT_lo, then Diag(gam) Vtilde as two bf16 terms
//   A2 = K^T [gV_hi | gV_lo]             (M d, N 2 NS, K 64)
//   S <- aC S + A2_hi + A2_lo            in fp32
//   QS = Q S_hi (M 64, N NS, K d) and AO = Att bf16(Vtilde) (M 64, N NS, K 64)
//   o  = scale Diag(D) QS + AO
// The state is an fp32 output, so no factor on its path may lose more than 16
// bits: S, Y, T and gam Vtilde enter the tensor cores as sums of two bf16 terms
// (2^-17 relative), K, Q and V are exact.  The two terms of a right operand sit
// side by side along N, where the second is nearly free: measured, a tcgen05.mma of
// K 16 takes 40 cycles at N 32, 48 at N 64, 64 at N 128, the same for M 64 as for
// M 128.  o is rounded to bf16 at the end, so its factors (S_hi, Att, Vtilde) are
// single bf16 terms.
//
// What bounds a chunk is the latency of the three rounds, product - epilogue -
// hand-off.  So
//  - the 64-row products are M = 64, whose rows lie 16 to a TMEM lane quadrant:
//    with the 16x256b load all 16 chain warps on all four SM sub-partitions share
//    the Y and Vtilde epilogues (M = 128 puts these rows on two quadrants, and
//    their epilogue took twice the time);
//  - the products beside the chain are issued where it waits: QS half under
//    the Y epilogue and half under the Vtilde epilogue, AO under the state's;
//  - the MMA warp runs converged and elects the issuing lane inside the
//    instruction, so that operands stay in uniform registers: eight products
//    are issued and complete in 512 cycles instead of 724;
//  - o and Vtilde leave by TMA stores from shared memory, not by the chain warps.
//
// Warps: 0 issues every tcgen05.mma, 1 every load (two chunks ahead); 16 chain
// warps (warp w: lane quadrant w % 4, one of four column groups) hold the state;
// 4 output warps.  Every wait is bounded as in the inter-chunk kernels of the
// momentum rule.
#include <cmath>

#include "gdr_tc.cuh"

namespace mdn {
namespace gdr {
namespace {

using namespace sm100;
using namespace tc;
using inter::wait_bar;
using inter::warp_wait;

constexpr int kChainWarp0 = 2, OW = 4;
constexpr int NVC = 4;  // slots of V and the record

template <int D, int NS>
struct Cfg {
    static constexpr int NH = NS == 16 ? 8 : NS / 4;  // columns of a chain thread's state
    static constexpr int CW = 4 * (NS / NH);          // chain warps
    static constexpr int kOutWarp0 = kChainWarp0 + CW;
    static constexpr int kThreads = (kOutWarp0 + OW) * 32;
    static constexpr int KP = D / 64;  // 64-column panels of K, Q
    static constexpr uint32_t KQ_BYTES = KP * 16384;
    static constexpr int NK = NS <= 32 ? 3 : 2;               // slots of K, Q and of T, Att
    static constexpr uint32_t KQ0 = 0;                        // [K; Q], NK slots
    static constexpr uint32_t FB0 = NK * KQ_BYTES;            // T_hi, Att, T_lo, NK slots
    static constexpr uint32_t ST = FB0 + NK * kBlkImg;        // [S_hi | S_lo], D rows, MN-major
    static constexpr uint32_t ST_BYTES = D * 2 * NS * 2;
    static constexpr uint32_t YB = ST + ST_BYTES;             // [Y_hi | Y_lo], then [gV_hi | gV_lo]
    static constexpr uint32_t V_BYTES = 64 * NS * 2;
    static constexpr uint32_t VB = YB + 2 * V_BYTES;          // bf16 Vtilde, MN-major
    static constexpr uint32_t OB = VB + V_BYTES;              // bf16 o, the same layout
    static constexpr uint32_t V0 = OB + V_BYTES;              // V slice, the same layout, NVC slots
    static constexpr uint32_t CR0 = V0 + NVC * V_BYTES;       // records
    static constexpr uint32_t BARS = CR0 + NVC * 1024;
    static constexpr uint32_t MISC = BARS + 288;
    static constexpr uint32_t BYTES = MISC + 16;
    static_assert(BYTES <= 232448, "shared memory");
    static constexpr uint32_t TM_KS = 0;             // 2 NS
    static constexpr uint32_t TM_AT = 2 * NS;        // 2 NS; A2 over it (AT is read before A2 is
    static constexpr uint32_t TM_A2 = TM_AT;         // issued, A2 before the next AT)
    static constexpr uint32_t TM_QS = 4 * NS;        // 2 slots x NS
    static constexpr uint32_t TM_AO = 6 * NS;        // 2 slots x NS
    static constexpr uint32_t kTmemCols = 8 * NS;
    // Right operands: rows of 2 NS x 2 bytes, hi and lo side by side (for NS 64 two panels),
    // swizzled by the row length; Vtilde, V and o have rows of half that.
    static constexpr uint32_t kSwY = NS == 16 ? kSw64 : kSw128, kSboY = NS == 16 ? 512 : 1024;
    static constexpr uint32_t kSwV = NS == 16 ? kSw32 : NS == 32 ? kSw64 : kSw128, kSboV = NS * 16;
    static constexpr uint32_t kRowStepY = NS == 16 ? 1024 : 2048;  // bytes of 16 rows (one panel)
    // 16-byte piece c (8 columns) of row i of the hi (lo = 0) or lo part of a right operand
    __device__ static __forceinline__ uint32_t off(int i, int c, int lo, uint32_t panel) {
        return NS == 16 ? sw64_off(i, 2 * lo + c) : NS == 32 ? sw128_off(i, 4 * lo + c)
                                                             : lo * panel + sw128_off(i, c);
    }
    __device__ static __forceinline__ uint32_t v_off(int r, int c) {
        return NS == 16 ? sw32_off(r, c) : NS == 32 ? sw64_off(r, c) : sw128_off(r, c);
    }
};

// mbarriers
constexpr int B_FKQ = 0;   // [3] K, Q landed
constexpr int B_FFB = 3;   // [3] T, Att landed
constexpr int B_KF = 6;    // [3] K, Q slot free (A2 complete, and A1, QS before it)
constexpr int B_FF = 9;    // [3] T, Att slot free (AO complete)
constexpr int B_FVC = 12;  // [4] V, record landed
constexpr int B_EVC = 16;  // [4] V, record slot read (chain and output warps)
constexpr int B_M1 = 20;   //     A1 complete
constexpr int B_MT = 21;   //     AT complete
constexpr int B_M2 = 22;   // [2] A2 complete
constexpr int B_MO = 24;   // [2] AO complete
constexpr int B_YR = 26;   //     Y written
constexpr int B_GR = 27;   //     gam Vtilde written
constexpr int B_VR = 28;   //     Vtilde written
constexpr int B_SR = 29;   //     next state written
constexpr int B_OD = 30;   // [2] QS, AO slot read by the output warps
constexpr int B_VF = 32;   //     Vtilde stored: its tile is free
constexpr int B_FIN = 33;
constexpr int kBars = 34;

struct ChainArgs {
    Args a;
    const uint8_t* blk;
    bool overlap;  // the operand kernel may still be running: wait for each block's flag
};

template <int N>
__device__ __forceinline__ void ld_cols(uint32_t t, float* v) {
    if constexpr (N == 8) tmem_ld8(t, v);
    else tmem_ld16(t, v);
}

template <int D, int NS>
__global__ void __launch_bounds__(Cfg<D, NS>::kThreads, 1)
chain_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
             const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
             const __grid_constant__ CUtensorMap tm_vt, const ChainArgs p)
{
    using L = Cfg<D, NS>;
    constexpr int NH = L::NH, NP = NH / 8;  // NP: 8-column pieces of a chain thread
    constexpr int CW = L::CW, kOutWarp0 = L::kOutWarp0, NK = L::NK;
    const Args& a = p.a;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, lid = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform
    const int quad = warp & 3;
    constexpr int SL = D / NS;
    const Chain ch = chain_of(a, blockIdx.x / SL);
    const int j0 = (blockIdx.x % SL) * NS;
    const int NT = (ch.len + kChunk - 1) / kChunk;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BARS);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC + 4);
    // token coordinates of the chain's first row in the TMA maps
    const int tb = a.cu_s ? 0 : (int)(ch.row0 / (a.T > 0 ? a.T : 1));
    const int tt0 = a.cu_s ? (int)ch.row0 : 0;

    if (tid == 0) {
        for (int k = 0; k < kBars; ++k) {
            uint32_t count = 1;
            if (k >= B_EVC && k < B_EVC + NVC) count = CW + OW;
            if (k >= B_YR && k <= B_SR) count = CW;
            if (k == B_OD || k == B_OD + 1 || k == B_VF) count = OW;
            mbar_init(&bars[k], count);
        }
        mbar_fence_init();
        *abort_flag = 0;
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, L::kTmemCols);
        tmem_relinquish();
    }
    const bool chain = warp >= kChainWarp0 && warp < kOutWarp0;
    const int hc = (warp - kChainWarp0) >> 2;  // column group
    // the state row of this lane: the row of A2 that its TMEM lane holds (M = d)
    const bool srow = D == 128 || lid < 16;
    const int irow = D == 128 ? quad * 32 + lid : quad * 16 + (lid & 15);
    float s[NH];
    auto put_state = [&]() {
        if (!srow) return;
#pragma unroll
        for (int c = 0; c < NP; ++c) {
            uint4 hi, lo;
            split8(s + 8 * c, hi, lo);
            const int cc = hc * NP + c;
            *reinterpret_cast<uint4*>(sm + L::ST + L::off(irow, cc, 0, D * 128)) = hi;
            *reinterpret_cast<uint4*>(sm + L::ST + L::off(irow, cc, 1, D * 128)) = lo;
        }
    };
    const size_t srow0 = ((size_t)ch.state * D + irow) * D + j0 + NH * hc;
    if (chain) {
#pragma unroll
        for (int j = 0; j < NH; j += 4) {
            const float4 x = a.S0 && srow ? *reinterpret_cast<const float4*>(a.S0 + srow0 + j)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
            s[j] = x.x; s[j + 1] = x.y; s[j + 2] = x.z; s[j + 3] = x.w;
        }
        put_state();
        fence_proxy_async_smem();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tq = tmem + (static_cast<uint32_t>(quad * 32) << 16);

    if (warp == 0) {
        // ------------------------------------------------------------ MMA issue (converged)
        const uint64_t d_k0 = smem_desc(sbase + L::KQ0, 16, 1024, kSw128);
        const uint64_t d_kt0 = smem_desc(sbase + L::KQ0, 16384, 1024, kSw128);  // MN-major
        const uint64_t d_st = smem_desc(sbase + L::ST, D * 128, L::kSboY, L::kSwY);
        const uint64_t d_fb0 = smem_desc(sbase + L::FB0, 16, 1024, kSw128);
        const uint64_t d_y = smem_desc(sbase + L::YB, 8192, L::kSboY, L::kSwY);
        const uint64_t d_v = smem_desc(sbase + L::VB, 64 * NS * 2, L::kSboV, L::kSwV);
        constexpr uint32_t ystep = L::kRowStepY >> 4;
        constexpr uint32_t vstep = (16 * NS * 2) >> 4;
        constexpr uint32_t id1 = idesc_bf16(64, 2 * NS, false, true);
        constexpr uint32_t id2 = idesc_bf16(D, 2 * NS, true, true);
        constexpr uint32_t ido = idesc_bf16(64, NS, false, true);
        constexpr int KS = D / 16;
        bool go = NT > 0 && warp_wait(&bars[B_FKQ], 0, abort_flag);
        for (int n = 0; n < NT && go; ++n) {
            const int s2 = n & 1;
            if (n >= 1 && !warp_wait(&bars[B_SR], (n - 1) & 1, abort_flag)) break;
            tc_fence_after_sync();
            const int sk = n % NK;
            const uint64_t dk = d_k0 + sk * (L::KQ_BYTES >> 4), dq = dk + (8192 >> 4);
            const uint64_t dfb = d_fb0 + sk * (kBlkImg >> 4);
            const uint32_t qs = tmem + L::TM_QS + NS * s2;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                mma_bf16_elect(tmem + L::TM_KS, dk + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4),
                               d_st + ks * ystep, id1, ks > 0);
            mma_commit_elect(&bars[B_M1]);
#pragma unroll
            for (int ks = 0; ks < KS / 2; ++ks)
                mma_bf16_elect(qs, dq + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4),
                               d_st + ks * ystep, ido, ks > 0);
            if (!warp_wait(&bars[B_FFB + sk], (n / NK) & 1, abort_flag)) break;
            if (!warp_wait(&bars[B_YR], n & 1, abort_flag)) break;
            tc_fence_after_sync();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_bf16_elect(tmem + L::TM_AT, dfb + ks * 2, d_y + ks * ystep, id1, ks > 0);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_bf16_elect(tmem + L::TM_AT, dfb + (kBlkTlo >> 4) + ks * 2, d_y + ks * ystep, id1, 1);
            mma_commit_elect(&bars[B_MT]);
#pragma unroll
            for (int ks = KS / 2; ks < KS; ++ks)
                mma_bf16_elect(qs, dq + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4),
                               d_st + ks * ystep, ido, 1);
            // what the next chunk's products need, while Vtilde is formed
            if (n + 1 < NT && !warp_wait(&bars[B_FKQ + (n + 1) % NK], ((n + 1) / NK) & 1, abort_flag)) break;
            if (n >= 1 && !warp_wait(&bars[B_OD + ((n + 1) & 1)], ((n - 1) >> 1) & 1, abort_flag)) break;
            if (!warp_wait(&bars[B_GR], n & 1, abort_flag)) break;
            tc_fence_after_sync();
            const uint64_t dkt = d_kt0 + sk * (L::KQ_BYTES >> 4);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_bf16_elect(tmem + L::TM_A2, dkt + ks * (2048 >> 4), d_y + ks * ystep, id2, ks > 0);
            mma_commit_elect(&bars[B_M2 + s2]);
            mma_commit_elect(&bars[B_KF + sk]);
            if (!warp_wait(&bars[B_VR], n & 1, abort_flag)) break;
            tc_fence_after_sync();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_bf16_elect(tmem + L::TM_AO + NS * s2, dfb + (kBlkAtt >> 4) + ks * 2, d_v + ks * vstep,
                               ido, ks > 0);
            mma_commit_elect(&bars[B_MO + s2]);
            mma_commit_elect(&bars[B_FF + sk]);
        }
        mma_commit_elect(&bars[B_FIN]);
        (void)mbar_wait(&bars[B_FIN], 0);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ loads
        if (lid == 0) {
            int done_kq = 0, done_fb = 0, done_vc = 0;
            for (int n = 0; n < NT; ++n) {
                const int sk = n % NK, sv = n % NVC;
                const size_t blk = (size_t)((ch.chunk0 + n) * a.H + ch.h) * kBlkBytes;
                const int t = tt0 + n * kChunk;
                if (n >= NK && !wait_bar(&bars[B_KF + sk], ((n / NK) - 1) & 1, abort_flag)) break;
                uint64_t* fb = &bars[B_FKQ + sk];
                mbar_arrive_expect_tx(fb, L::KQ_BYTES);
#pragma unroll
                for (int q = 0; q < L::KP; ++q) {
                    uint8_t* dst = sm + L::KQ0 + sk * L::KQ_BYTES + q * 16384;
                    tma_load_4d(dst, &tm_k, q * 64, ch.hk, t, tb, fb);
                    tma_load_4d(dst + 8192, &tm_q, q * 64, ch.hk, t, tb, fb);
                }
                done_kq = n + 1;
                if (n >= NVC && !wait_bar(&bars[B_EVC + sv], ((n / NVC) - 1) & 1, abort_flag)) break;
                // the chunk's block is in global memory (its kernel may still be running)
                if (p.overlap) {
                    if (!inter::wait_ready(a.ready + (ch.chunk0 + n) * a.H + ch.h, abort_flag)) break;
                    fence_proxy_async_global();
                }
                fb = &bars[B_FVC + sv];
                mbar_arrive_expect_tx(fb, L::V_BYTES + 1024);
                tma_load_4d(sm + L::V0 + sv * L::V_BYTES, &tm_v, j0, ch.h, t, tb, fb);
                bulk_load(sm + L::CR0 + sv * 1024, p.blk + blk + kBlkRec, 1024, fb);
                done_vc = n + 1;
                if (n >= NK && !wait_bar(&bars[B_FF + sk], ((n / NK) - 1) & 1, abort_flag)) break;
                fb = &bars[B_FFB + sk];
                mbar_arrive_expect_tx(fb, kBlkImg);
                bulk_load(sm + L::FB0 + sk * kBlkImg, p.blk + blk, kBlkImg, fb);
                done_fb = n + 1;
            }
            // copies in flight must land before shared memory is released
            for (int n = done_kq - NK; n < done_kq; ++n)
                if (n >= 0) (void)mbar_wait(&bars[B_FKQ + n % NK], (n / NK) & 1);
            for (int n = done_fb - NK; n < done_fb; ++n)
                if (n >= 0) (void)mbar_wait(&bars[B_FFB + n % NK], (n / NK) & 1);
            for (int n = done_vc - NVC; n < done_vc; ++n)
                if (n >= 0) (void)mbar_wait(&bars[B_FVC + n % NVC], (n / NVC) & 1);
        }
        __syncwarp();
    } else if (chain) {
        // ------------------------------------------------------------ chain epilogues
        // Y, Vtilde: rows r0, r0 + 8 of the 16 of this quadrant, columns c0, c0 + 1 of
        // each 8-column piece (the 16x256b layout)
        const int r0 = quad * 16 + (lid >> 2), pc = (lid & 3) * 4;  // pc: byte of the column pair
        for (int n = 0; n < NT; ++n) {
            const int s2 = n & 1, sv = n % NVC;
            const int valid = ch.len - n * kChunk;  // tokens from this chunk's first on
            if (!warp_wait(&bars[B_FVC + sv], (n / NVC) & 1, abort_flag)) break;
            const float* cr = reinterpret_cast<const float*>(sm + L::CR0 + sv * 1024);
            const float aC = cr[kRecB];
            const float dr[2] = {cr[kRecD + r0], cr[kRecD + r0 + 8]};
            const float gr[2] = {cr[kRecGam + r0], cr[kRecGam + r0 + 8]};
            uint32_t vw[NP][2];
#pragma unroll
            for (int c = 0; c < NP; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    vw[c][e] = *reinterpret_cast<const uint32_t*>(sm + L::V0 + sv * L::V_BYTES +
                                                                  L::v_off(r0 + 8 * e, hc * NP + c) + pc);
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_EVC + sv]);
            if (valid < kChunk && a.cu_s) {
                // K rows behind the sequence belong to the next one (or to none) and
                // may hold anything: they meet zeros in A2, so make them zero
                if (!warp_wait(&bars[B_FKQ + n % NK], (n / NK) & 1, abort_flag)) break;
                for (int e = (warp - kChainWarp0) * 32 + lid; e < 64 * 8 * L::KP; e += CW * 32) {
                    const int r = e / (8 * L::KP), q = e % (8 * L::KP);
                    if (r >= valid)
                        *reinterpret_cast<uint4*>(sm + L::KQ0 + (n % NK) * L::KQ_BYTES + (q >> 3) * 16384 +
                                                  sw128_off(r, q & 7)) = make_uint4(0, 0, 0, 0);
                }
            }
            if (!warp_wait(&bars[B_M1], n & 1, abort_flag)) break;
            tc_fence_after_sync();
            float x[NP * 4], y[NP * 4];
            tmem_ld_16x256<NP>(tq + L::TM_KS + NH * hc, x);
            tmem_ld_16x256<NP>(tq + L::TM_KS + NS + NH * hc, y);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < NP; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 4 * c + 2 * e;
                    float v0, v1;
                    unpack2(vw[c][e], v0, v1);
                    v0 = fmaf(-dr[e], x[i] + y[i], v0);
                    v1 = fmaf(-dr[e], x[i + 1] + y[i + 1], v1);
                    if (r0 + 8 * e >= valid) v0 = v1 = 0.f;  // rows behind the sequence, whatever they hold
                    uint32_t hi, lo;
                    split2(v0, v1, hi, lo);
                    const int r = r0 + 8 * e, cc = hc * NP + c;
                    *reinterpret_cast<uint32_t*>(sm + L::YB + L::off(r, cc, 0, 8192) + pc) = hi;
                    *reinterpret_cast<uint32_t*>(sm + L::YB + L::off(r, cc, 1, 8192) + pc) = lo;
                }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_YR]);
            // the last chunk's Vtilde has left (its store was issued a chunk ago)
            if (n >= 1 && !warp_wait(&bars[B_VF], (n - 1) & 1, abort_flag)) break;
            if (!warp_wait(&bars[B_MT], n & 1, abort_flag)) break;
            tc_fence_after_sync();
            tmem_ld_16x256<NP>(tq + L::TM_AT + NH * hc, x);
            tmem_ld_16x256<NP>(tq + L::TM_AT + NS + NH * hc, y);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < NP; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 4 * c + 2 * e, r = r0 + 8 * e, cc = hc * NP + c;
                    x[i] += y[i];
                    x[i + 1] += y[i + 1];
                    uint32_t hi, lo;
                    split2(gr[e] * x[i], gr[e] * x[i + 1], hi, lo);
                    *reinterpret_cast<uint32_t*>(sm + L::YB + L::off(r, cc, 0, 8192) + pc) = hi;
                    *reinterpret_cast<uint32_t*>(sm + L::YB + L::off(r, cc, 1, 8192) + pc) = lo;
                }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_GR]);
#pragma unroll
            for (int c = 0; c < NP; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<uint32_t*>(sm + L::VB + L::v_off(r0 + 8 * e, hc * NP + c) + pc) =
                        pack_bf16(x[4 * c + 2 * e], x[4 * c + 2 * e + 1]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_VR]);
            if (!warp_wait(&bars[B_M2 + s2], (n >> 1) & 1, abort_flag)) break;
            tc_fence_after_sync();
            {
                float u[NH], w[NH];
                ld_cols<NH>(tq + L::TM_A2 + NH * hc, u);
                ld_cols<NH>(tq + L::TM_A2 + NS + NH * hc, w);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < NH; ++j) s[j] = fmaf(aC, s[j], u[j] + w[j]);
            }
            put_state();
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_SR]);
        }
    } else {
        // ------------------------------------------------------------ outputs
        // A warp's 16 rows are its own, in the tiles and in the stores, so that no barrier
        // joins the output warps.
        const int r0 = lid >> 2, pc = (lid & 3) * 4, w0 = quad * 16;
        constexpr uint32_t kStrip = 16 * NS * 2;
        // rows < valid of the warp's strip to global memory (a packed sequence's last
        // chunk: a TMA store would write into the next sequence)
        auto store_rows = [&](const uint8_t* tile, void* out, int n, int valid) {
            for (int e = lid; e < 16 * (NS / 8); e += 32) {
                const int r = w0 + e / (NS / 8), c = e % (NS / 8);
                if (r < valid)
                    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) +
                                              ((size_t)(ch.row0 + n * kChunk + r) * a.H + ch.h) * D + j0 + 8 * c) =
                        *reinterpret_cast<const uint4*>(tile + L::v_off(r, c));
            }
        };
        for (int n = 0; n < NT; ++n) {
            const int s2 = n & 1, sv = n % NVC;
            const int valid = min(kChunk, ch.len - n * kChunk);
            const bool whole = !a.cu_s || valid == kChunk;
            if (!warp_wait(&bars[B_FVC + sv], (n / NVC) & 1, abort_flag)) break;
            const float* cr = reinterpret_cast<const float*>(sm + L::CR0 + sv * 1024);
            const float dq[2] = {cr[kRecDq + w0 + r0], cr[kRecDq + w0 + r0 + 8]};
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_EVC + sv]);
            if (!warp_wait(&bars[B_VR], n & 1, abort_flag)) break;
            if (a.vt && !whole) store_rows(sm + L::VB, a.vt, n, valid);
            if (lid == 0) {
                if (a.vt && whole) {
                    tma_store_4d(&tm_vt, j0, ch.h, tt0 + n * kChunk + w0, tb, sm + L::VB + quad * kStrip);
                    bulk_commit_group();
                }
                bulk_wait_group_read<0>();  // Vtilde, and the o of the chunk before
                mbar_arrive(&bars[B_VF]);
            }
            __syncwarp();
            if (!warp_wait(&bars[B_MO + s2], (n >> 1) & 1, abort_flag)) break;
            tc_fence_after_sync();
            float x[NS / 2], y[NS / 2];
            tmem_ld_16x256<NS / 8>(tq + L::TM_QS + NS * s2, x);
            tmem_ld_16x256<NS / 8>(tq + L::TM_AO + NS * s2, y);
            tmem_wait_ld();
            tc_fence_before_sync();
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_OD + s2]);
#pragma unroll
            for (int c = 0; c < NS / 8; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<uint32_t*>(sm + L::OB + L::v_off(w0 + r0 + 8 * e, c) + pc) =
                        pack_bf16(fmaf(dq[e], x[4 * c + 2 * e], y[4 * c + 2 * e]),
                                  fmaf(dq[e], x[4 * c + 2 * e + 1], y[4 * c + 2 * e + 1]));
            fence_proxy_async_smem();
            __syncwarp();
            if (!whole) store_rows(sm + L::OB, a.o, n, valid);
            else if (lid == 0) {
                tma_store_4d(&tm_o, j0, ch.h, tt0 + n * kChunk + w0, tb, sm + L::OB + quad * kStrip);
                bulk_commit_group();
            }
        }
        if (lid == 0) bulk_wait_group_all();
    }

    // a call that follows may clear the work counter: not before the operand kernel is done
    if (p.overlap) pdl_wait();
    tc_fence_before_sync();
    __syncthreads();
    const bool ok = *abort_flag == 0;
    if (chain && ok && srow) {
#pragma unroll
        for (int j = 0; j < NH; j += 4)
            *reinterpret_cast<float4*>(a.S_T + srow0 + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
    }
    if (!ok && tid == 0) atomicOr(a.status + 1, 1u);
    if (warp == 0) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

template <int D, int NS>
cudaError_t launch_chain(const Args& a, bool overlap, cudaStream_t s)
{
    using L = Cfg<D, NS>;
    CUtensorMap mq, mk, mv, mo, mvt;
    const auto sw = NS == 16   ? CU_TENSOR_MAP_SWIZZLE_32B
                    : NS == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                               : CU_TENSOR_MAP_SWIZZLE_128B;
    if (!make_rows_map(&mq, a.q, a, a.Hk, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_rows_map(&mk, a.k, a, a.Hk, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_rows_map(&mv, a.v, a, a.H, NS, sw) ||
        !make_rows_map(&mo, a.o, a, a.H, NS, sw, 16) ||
        !make_rows_map(&mvt, a.vt ? a.vt : a.o, a, a.H, NS, sw, 16))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(chain_kernel<D, NS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)L::BYTES);
    if (e != cudaSuccess) return e;
    ChainArgs p{a, a.blk, overlap};
    ProfScope ps(kGdrChain, s);
    if (!overlap) {
        chain_kernel<D, NS><<<(unsigned)(chains(a) * (D / NS)), L::kThreads, L::BYTES, s>>>(mq, mk, mv, mo, mvt, p);
        return cudaGetLastError();
    }
    return launch_dependent(chain_kernel<D, NS>, (unsigned)(chains(a) * (D / NS)), L::kThreads, (size_t)L::BYTES, s,
                            mq, mk, mv, mo, mvt, p);
}

}  // namespace

// Chain width.  A chunk's step takes 1.23, 1.65 and 2.4 us with 16, 32 and 64 columns per
// CTA (measured, 4096 tokens): the narrowest slice whose CTAs all fit on the SMs at once
// has the shortest chain; beyond that the widest, which takes the least SM time per chunk
// of a head of d 128 (4.8 us against 6.6 and 9.8).  16384 tokens of 16 heads: 287 us in
// slices of 16, 374 of 32, 447 of 64.  Packed sequences start longest first (the longest chain is the
// critical path), so they keep 32 columns up to four waves.
//
// The chain is launched as the operand kernel's programmatic dependent.  Its CTAs need
// a whole SM, so the operand CTAs on as many SMs as the chain's CTAs leave over beside
// whole waves stop after L chunks each, and those on the other SMs (U of them) make the
// rest, which the work order makes the chunks the chains need last; the chain's first,
// partial wave runs meanwhile.  With r chain steps per operand chunk (11k cycles at three
// CTAs an SM), L minimises  L r + max(NT, rest / U r + 1).  Measured, operands and chain:
// 16384 tokens of 16 heads 350 -> 308 us, packed sequences of 1 to 24576 tokens 792 -> 683,
// 4 x 2048 tokens of 8 heads 84 -> 77, 8 x 4096 of 16 (256 CTAs) 416 -> 393 (in a loop of
// seconds, at the power cap, 411 to 415).  Whole waves
// only: nothing is reserved and nothing overlaps.
cudaError_t launch_fwd_tc(const Args& a, cudaStream_t s)
{
    int dev = 0, sms = 148;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    const long long n = chains(a);
    const int ns = a.D == 64 ? (n * 4 <= sms ? 16 : 32)
                   : n * 8 <= sms ? 16
                   : n * 4 <= (a.cu_s ? 4 * sms : sms) ? 32 : 64;
    const long long ctas = n * (a.D / ns);
    int reserve = 0, limit = 1;
    if (a.cu_s) {
        // packed: SMs from the start for the chains of the longest sequence
        const long long first = (long long)a.H * (a.D / ns), room = sms - sms / 4;
        reserve = (int)(first < ctas ? (first < room ? first : room) : (ctas < room ? ctas : room));
    } else if (ctas % sms) {
        const double r = ns == 16 ? 5.0 : ns == 32 ? 3.9 : 2.5;
        const long long first = ctas % sms;
        const long long U = 3LL * (sms - first), round = 3LL * sms, total = chunks(a) * a.H;
        double best = 0.0;
        for (int L = 1; (L - 1) * round < total; ++L) {
            const long long rest = total - L * round;
            const double t = L * r + (rest > 0 ? fmax((double)a.NT, (double)rest / U * r + 1.0) : (double)a.NT);
            if (L == 1 || t < best) {
                best = t;
                reserve = (int)first;
                limit = L;
            }
        }
    }
    if ((e = launch_operands_tc(a, s, false, reserve, limit)) != cudaSuccess) return e;
    const bool over = reserve > 0;
    if (a.D == 64) return ns == 16 ? launch_chain<64, 16>(a, over, s) : launch_chain<64, 32>(a, over, s);
    return ns == 16   ? launch_chain<128, 16>(a, over, s)
           : ns == 32 ? launch_chain<128, 32>(a, over, s)
                      : launch_chain<128, 64>(a, over, s);
}

}  // namespace gdr
}  // namespace mdn
