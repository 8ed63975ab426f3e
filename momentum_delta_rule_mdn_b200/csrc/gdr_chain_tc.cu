// The forward chain of the gated delta rule on sm_100a (formulas in gdr_tc.cuh):
// one CTA per chain and NS of its d_v columns, walking the chunks in order with
// the state in fp32 registers.
//
// Per chunk, three dependent rounds on the tensor cores and one beside them:
//   A1 = [K; Q] [S_hi | S_lo]            (M 128, N 2 NS, K d)
//   Y  = V - Diag(D) K (S_hi + S_lo)     in fp32, as two bf16 terms
//   AT = T_hi [Y_hi | Y_lo] + T_lo [Y_hi | Y_lo]    (M 128, N 2 NS, K 64)
//   Vtilde = AT_hi + AT_lo, then Diag(gam) Vtilde as two bf16 terms
//   A2 = K^T [gV_hi | gV_lo]             (M 128, N 2 NS, K 64; K^T is the K tile
//                                         read MN-major)
//   S <- aC S + A2_hi + A2_lo            in fp32
//   AO = Att bf16(Vtilde)                (M 128, N NS, K 64), beside the state update
//   o  = scale Diag(D) Q S_hi + AO
// The state is an fp32 output, so no factor on its path may lose more than 16
// bits: S, Y, T and gam Vtilde enter the tensor cores as sums of two bf16 terms
// (2^-17 relative), K, Q and V are exact.  The two terms of a right operand sit
// side by side along N, where they cost nothing: a tcgen05.mma of N <= 128 takes
// the same time whatever N is.  o is rounded to bf16 at the end, so its
// factors (S_hi, Att, Vtilde) are single bf16 terms.
//
// Warps: 0 issues every tcgen05.mma, 1 every load (two chunks ahead); 16 chain
// warps hold the state, warp w the TMEM lanes 32 (w % 4) .. and one of four
// column groups, those on lanes 0..63 (the K rows) also form Y and Vtilde and
// store Vtilde; 2 output warps on lanes 64..127 (the Q rows) form and store o.
// Every wait is bounded as in the inter-chunk kernels of the momentum rule.
#include "gdr_tc.cuh"

namespace mdn {
namespace gdr {
namespace {

using namespace sm100;
using namespace tc;
using inter::wait_bar;
using inter::warp_wait;

constexpr int kChainWarp0 = 2, CW = 16, kOutWarp0 = kChainWarp0 + CW, kThreads = (kOutWarp0 + 2) * 32;
constexpr int NVC = 4;  // slots of V and the record

template <int D, int NS>
struct Cfg {
    static constexpr int NH = NS / 4;  // columns of a chain thread
    static constexpr int KP = D / 64;  // 64-column panels of K, Q
    static constexpr uint32_t KQ_BYTES = KP * 16384;
    static constexpr uint32_t KQ0 = 0;                        // [K; Q], 2 slots
    static constexpr uint32_t FB0 = 2 * KQ_BYTES;             // [T_hi; Att], T_lo, 2 slots
    static constexpr uint32_t ST = FB0 + 2 * kBlkImg;         // [S_hi | S_lo], D rows, MN-major
    static constexpr uint32_t ST_BYTES = 128 * 2 * NS * 2;
    static constexpr uint32_t YB = ST + ST_BYTES;             // [Y_hi | Y_lo], then [gV_hi | gV_lo]
    static constexpr uint32_t VB = YB + 64 * 2 * NS * 2;      // bf16 Vtilde, MN-major
    static constexpr uint32_t V0 = VB + 64 * NS * 2;          // V slice, plain rows, NVC slots
    static constexpr uint32_t V_BYTES = 64 * NS * 2;
    static constexpr uint32_t CR0 = V0 + NVC * V_BYTES;       // records
    static constexpr uint32_t BARS = CR0 + NVC * 1024;
    static constexpr uint32_t MISC = BARS + 256;
    static constexpr uint32_t BYTES = MISC + 16;
    static_assert(BYTES <= 232448, "shared memory");
    // the M = 128 operand at T_lo reads 8 KB behind it (lanes 64..127, unused)
    static constexpr uint32_t TM_A1 = 0;             // 2 slots x 2 NS
    static constexpr uint32_t TM_AT = 4 * NS;        // 2 NS
    static constexpr uint32_t TM_A2 = TM_AT;         // AT is read before A2 is issued, and A2 before the next AT
    static constexpr uint32_t TM_AO = 6 * NS;        // 2 slots x NS
    static constexpr uint32_t kTmemCols = 8 * NS;
    // 16-byte piece c (8 columns) of row i of the hi (lo = 0) or lo part of a right operand
    __device__ static __forceinline__ uint32_t off(int i, int c, int lo, uint32_t panel) {
        return NS == 32 ? sw128_off(i, 4 * lo + c) : lo * panel + sw128_off(i, c);
    }
    __device__ static __forceinline__ uint32_t v_off(int r, int c) {
        return NS == 32 ? sw64_off(r, c) : sw128_off(r, c);
    }
};

// mbarriers
constexpr int B_FKQ = 0;   // [2] K, Q landed
constexpr int B_FFB = 2;   // [2] T, Att landed
constexpr int B_FVC = 4;   // [4] V, record landed
constexpr int B_EVC = 8;   // [4] V, record slot read (chain and output warps)
constexpr int B_M1 = 12;   // [2] A1 complete
constexpr int B_MT = 14;   //     AT complete
constexpr int B_M2 = 15;   // [2] A2 complete (and A1: the K, Q slot is free)
constexpr int B_MO = 17;   // [2] AO complete (the T, Att slot is free)
constexpr int B_YR = 19;   //     Y written
constexpr int B_GR = 20;   //     gam Vtilde written (all chain warps: see the K rows past the end)
constexpr int B_VR = 21;   //     Vtilde written
constexpr int B_SR = 22;   //     next state written
constexpr int B_OD = 23;   // [2] A1, AO slot read by the output warps
constexpr int B_FIN = 25;
constexpr int kBars = 26;

struct ChainArgs {
    Args a;
    const uint8_t* blk;
};

template <int N>
__device__ __forceinline__ void ld_cols(uint32_t t, float* v) {
    if constexpr (N == 8) tmem_ld8(t, v);
    else tmem_ld16(t, v);
}

template <int D, int NS>
__global__ void __launch_bounds__(kThreads, 1)
chain_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
             const __grid_constant__ CUtensorMap tm_v, const ChainArgs p)
{
    using L = Cfg<D, NS>;
    constexpr int NH = L::NH;
    const Args& a = p.a;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lid = tid & 31;
    const int quad = warp & 3, lane = (quad << 5) | lid;
    constexpr int SL = D / NS;
    const Chain ch = chain_of(a, blockIdx.x / SL);
    const int j0 = (blockIdx.x % SL) * NS;
    const int NT = (ch.len + kChunk - 1) / kChunk;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BARS);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC + 4);

    if (tid == 0) {
        for (int k = 0; k < kBars; ++k) {
            uint32_t count = 1;
            if (k >= B_EVC && k < B_EVC + NVC) count = CW + 2;
            if (k == B_YR || k == B_VR) count = CW / 2;
            if (k == B_GR || k == B_SR) count = CW;
            if (k == B_OD || k == B_OD + 1) count = 2;
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
    const bool srow = lane < D;                // this lane is a row of S
    float s[NH];
    auto put_state = [&]() {
        if (!srow) return;
#pragma unroll
        for (int c = 0; c < NH / 8; ++c) {
            uint4 hi, lo;
            split8(s + 8 * c, hi, lo);
            const int cc = hc * (NH / 8) + c;
            *reinterpret_cast<uint4*>(sm + L::ST + L::off(lane, cc, 0, 16384)) = hi;
            *reinterpret_cast<uint4*>(sm + L::ST + L::off(lane, cc, 1, 16384)) = lo;
        }
    };
    const size_t srow0 = ((size_t)ch.state * D + lane) * D + j0 + NH * hc;
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
        // ------------------------------------------------------------ MMA issue
        if (lid == 0) {
            const uint64_t d_kq0 = smem_desc(sbase + L::KQ0, 16, 1024, kSw128);
            // K^T: the K rows read MN-major (64-column panels 16 KB apart)
            const uint64_t d_kt0 = smem_desc(sbase + L::KQ0, 16384, 1024, kSw128);
            const uint64_t d_st = smem_desc(sbase + L::ST, 16384, 1024, kSw128);
            const uint64_t d_fb0 = smem_desc(sbase + L::FB0, 16, 1024, kSw128);
            const uint64_t d_y = smem_desc(sbase + L::YB, 8192, 1024, kSw128);
            const uint64_t d_v = NS == 32 ? smem_desc(sbase + L::VB, 4096, 512, kSw64)
                                          : smem_desc(sbase + L::VB, 8192, 1024, kSw128);
            constexpr uint32_t vstep = (16 * NS * 2) >> 4;
            constexpr uint32_t id1 = idesc_bf16(128, 2 * NS, false, true);
            constexpr uint32_t id2 = idesc_bf16(128, 2 * NS, true, true);
            constexpr uint32_t ido = idesc_bf16(128, NS, false, true);
            bool ready = NT > 0 && wait_bar(&bars[B_FKQ], 0, abort_flag);
            for (int n = 0; n < NT && ready; ++n) {
                const int s2 = n & 1;
                if (n >= 1 && !wait_bar(&bars[B_SR], (n - 1) & 1, abort_flag)) break;
                tc_fence_after_sync();
                const uint64_t dkq = d_kq0 + s2 * (L::KQ_BYTES >> 4);
                const uint32_t a1 = tmem + L::TM_A1 + 2 * NS * s2;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_bf16(a1, dkq + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4),
                             d_st + ks * (2048 >> 4), id1, ks > 0);
                mma_commit(&bars[B_M1 + s2]);
                if (!wait_bar(&bars[B_FFB + s2], (n >> 1) & 1, abort_flag)) break;
                if (!wait_bar(&bars[B_YR], n & 1, abort_flag)) break;
                tc_fence_after_sync();
                const uint64_t dfb = d_fb0 + s2 * (kBlkImg >> 4);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16(tmem + L::TM_AT, dfb + ks * 2, d_y + ks * (2048 >> 4), id1, ks > 0);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16(tmem + L::TM_AT, dfb + (kBlkTlo >> 4) + ks * 2, d_y + ks * (2048 >> 4), id1, 1);
                mma_commit(&bars[B_MT]);
                // what the next A1 and this AO need, while Vtilde is formed
                if (n + 1 < NT && !wait_bar(&bars[B_FKQ + ((n + 1) & 1)], ((n + 1) >> 1) & 1, abort_flag)) break;
                if (n >= 1 && !wait_bar(&bars[B_OD + ((n + 1) & 1)], ((n - 1) >> 1) & 1, abort_flag)) break;
                if (!wait_bar(&bars[B_GR], n & 1, abort_flag)) break;
                tc_fence_after_sync();
                const uint64_t dkt = d_kt0 + s2 * (L::KQ_BYTES >> 4);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16(tmem + L::TM_A2, dkt + ks * (2048 >> 4), d_y + ks * (2048 >> 4), id2, ks > 0);
                mma_commit(&bars[B_M2 + s2]);
                if (!wait_bar(&bars[B_VR], n & 1, abort_flag)) break;
                tc_fence_after_sync();
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16(tmem + L::TM_AO + NS * s2, dfb + ks * 2, d_v + ks * vstep, ido, ks > 0);
                mma_commit(&bars[B_MO + s2]);
            }
            mma_commit(&bars[B_FIN]);
            (void)mbar_wait(&bars[B_FIN], 0);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ loads
        if (lid == 0) {
            int done_kq = 0, done_fb = 0, done_vc = 0;
            const int b = a.cu_s ? 0 : (int)(ch.row0 / (a.T > 0 ? a.T : 1));
            const int t0 = a.cu_s ? (int)ch.row0 : 0;
            for (int n = 0; n < NT; ++n) {
                const int s2 = n & 1, sv = n % NVC;
                const size_t blk = (size_t)((ch.chunk0 + n) * a.H + ch.h) * kBlkBytes;
                const int t = t0 + n * kChunk;
                if (n >= 2 && !wait_bar(&bars[B_M2 + s2], ((n - 2) >> 1) & 1, abort_flag)) break;
                uint64_t* fb = &bars[B_FKQ + s2];
                mbar_arrive_expect_tx(fb, L::KQ_BYTES);
#pragma unroll
                for (int q = 0; q < L::KP; ++q) {
                    uint8_t* dst = sm + L::KQ0 + s2 * L::KQ_BYTES + q * 16384;
                    tma_load_4d(dst, &tm_k, q * 64, ch.hk, t, b, fb);
                    tma_load_4d(dst + 8192, &tm_q, q * 64, ch.hk, t, b, fb);
                }
                done_kq = n + 1;
                if (n >= NVC && !wait_bar(&bars[B_EVC + sv], ((n / NVC) - 1) & 1, abort_flag)) break;
                fb = &bars[B_FVC + sv];
                mbar_arrive_expect_tx(fb, L::V_BYTES + 1024);
                tma_load_4d(sm + L::V0 + sv * L::V_BYTES, &tm_v, j0, ch.h, t, b, fb);
                bulk_load(sm + L::CR0 + sv * 1024, p.blk + blk + kBlkRec, 1024, fb);
                done_vc = n + 1;
                if (n >= 2 && !wait_bar(&bars[B_MO + s2], ((n - 2) >> 1) & 1, abort_flag)) break;
                fb = &bars[B_FFB + s2];
                mbar_arrive_expect_tx(fb, kBlkImg);
                bulk_load(sm + L::FB0 + s2 * kBlkImg, p.blk + blk, kBlkImg, fb);
                done_fb = n + 1;
            }
            // copies in flight must land before shared memory is released
            for (int n = done_kq - 2; n < done_kq; ++n)
                if (n >= 0) (void)mbar_wait(&bars[B_FKQ + (n & 1)], (n >> 1) & 1);
            for (int n = done_fb - 2; n < done_fb; ++n)
                if (n >= 0) (void)mbar_wait(&bars[B_FFB + (n & 1)], (n >> 1) & 1);
            for (int n = done_vc - NVC; n < done_vc; ++n)
                if (n >= 0) (void)mbar_wait(&bars[B_FVC + n % NVC], (n / NVC) & 1);
        }
        __syncwarp();
    } else if (chain) {
        // ------------------------------------------------------------ chain epilogues
        const bool ypart = quad < 2;
        const int r = lane & 63;
        for (int n = 0; n < NT; ++n) {
            const int s2 = n & 1, sv = n % NVC;
            const int valid = ch.len - n * kChunk;  // tokens from this chunk's first on
            if (!warp_wait(&bars[B_FVC + sv], (n / NVC) & 1, abort_flag)) break;
            const float* cr = reinterpret_cast<const float*>(sm + L::CR0 + sv * 1024);
            const float aC = cr[kRecB];
            if (ypart) {
                const float dr = cr[kRecD + r], gr = cr[kRecGam + r];
                const uint4* vrow = reinterpret_cast<const uint4*>(sm + L::V0 + sv * L::V_BYTES + r * (NS * 2)) +
                                    hc * (NH / 8);
                uint4 vw[NH / 8];
#pragma unroll
                for (int c = 0; c < NH / 8; ++c) vw[c] = vrow[c];
                __syncwarp();
                if (lid == 0) mbar_arrive(&bars[B_EVC + sv]);
                if (!warp_wait(&bars[B_M1 + s2], (n >> 1) & 1, abort_flag)) break;
                tc_fence_after_sync();
                float x[NH], y[NH];
                ld_cols<NH>(tq + L::TM_A1 + 2 * NS * s2 + NH * hc, x);
                ld_cols<NH>(tq + L::TM_A1 + 2 * NS * s2 + NS + NH * hc, y);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < NH / 8; ++c) {
                    float vv[8];
                    unpack_bf16x8(vw[c], vv);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        vv[e] = fmaf(-dr, x[8 * c + e] + y[8 * c + e], vv[e]);
                        if (r >= valid) vv[e] = 0.f;  // rows behind the sequence, whatever they hold
                    }
                    uint4 hi, lo;
                    split8(vv, hi, lo);
                    const int cc = hc * (NH / 8) + c;
                    *reinterpret_cast<uint4*>(sm + L::YB + L::off(r, cc, 0, 8192)) = hi;
                    *reinterpret_cast<uint4*>(sm + L::YB + L::off(r, cc, 1, 8192)) = lo;
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lid == 0) mbar_arrive(&bars[B_YR]);
                if (!warp_wait(&bars[B_MT], n & 1, abort_flag)) break;
                tc_fence_after_sync();
                ld_cols<NH>(tq + L::TM_AT + NH * hc, x);
                ld_cols<NH>(tq + L::TM_AT + NS + NH * hc, y);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < NH; ++j) {
                    x[j] += y[j];
                    y[j] = gr * x[j];
                }
#pragma unroll
                for (int c = 0; c < NH / 8; ++c) {
                    uint4 hi, lo;
                    split8(y + 8 * c, hi, lo);
                    const int cc = hc * (NH / 8) + c;
                    *reinterpret_cast<uint4*>(sm + L::YB + L::off(r, cc, 0, 8192)) = hi;
                    *reinterpret_cast<uint4*>(sm + L::YB + L::off(r, cc, 1, 8192)) = lo;
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lid == 0) mbar_arrive(&bars[B_GR]);
#pragma unroll
                for (int c = 0; c < NH / 8; ++c) {
                    vw[c] = bf16x8(x + 8 * c);
                    *reinterpret_cast<uint4*>(sm + L::VB + L::v_off(r, hc * (NH / 8) + c)) = vw[c];
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lid == 0) mbar_arrive(&bars[B_VR]);
                if (a.vt && r < valid) {
                    uint4* dst = reinterpret_cast<uint4*>(
                        static_cast<__nv_bfloat16*>(a.vt) +
                        ((size_t)(ch.row0 + n * kChunk + r) * a.H + ch.h) * D + j0 + NH * hc);
#pragma unroll
                    for (int c = 0; c < NH / 8; ++c) dst[c] = vw[c];
                }
            } else {
                __syncwarp();
                if (lid == 0) mbar_arrive(&bars[B_EVC + sv]);
                if (valid < kChunk && a.cu_s) {
                    // K rows behind the sequence belong to the next one (or to none)
                    // and may hold anything: they meet zeros in A2, so make them zero
                    if (!warp_wait(&bars[B_FKQ + s2], (n >> 1) & 1, abort_flag)) break;
                    if (r >= valid)
#pragma unroll
                        for (int c = 0; c < 2 * L::KP; ++c) {
                            const int q = hc * 2 * L::KP + c;  // 16-byte piece of the row
                            *reinterpret_cast<uint4*>(sm + L::KQ0 + s2 * L::KQ_BYTES + (q >> 3) * 16384 +
                                                      sw128_off(r, q & 7)) = make_uint4(0, 0, 0, 0);
                        }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lid == 0) mbar_arrive(&bars[B_GR]);
            }
            if (!warp_wait(&bars[B_M2 + s2], (n >> 1) & 1, abort_flag)) break;
            tc_fence_after_sync();
            {
                float x[NH], y[NH];
                ld_cols<NH>(tq + L::TM_A2 + NH * hc, x);
                ld_cols<NH>(tq + L::TM_A2 + NS + NH * hc, y);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < NH; ++j) s[j] = fmaf(aC, s[j], x[j] + y[j]);
            }
            put_state();
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_SR]);
        }
    } else {
        // ------------------------------------------------------------ outputs (lanes 64..127)
        const int r = lane & 63;
        for (int n = 0; n < NT; ++n) {
            const int s2 = n & 1, sv = n % NVC;
            if (!warp_wait(&bars[B_FVC + sv], (n / NVC) & 1, abort_flag)) break;
            const float dq = reinterpret_cast<const float*>(sm + L::CR0 + sv * 1024)[kRecDq + r];
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_EVC + sv]);
            if (!warp_wait(&bars[B_MO + s2], (n >> 1) & 1, abort_flag)) break;
            tc_fence_after_sync();
            const int t = n * kChunk + r;
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) +
                                                  ((size_t)(ch.row0 + t) * a.H + ch.h) * D + j0);
#pragma unroll 1
            for (int q = 0; q < NS / 16; ++q) {
                float x[16], y[16];
                tmem_ld16(tq + L::TM_A1 + 2 * NS * s2 + 16 * q, x);
                tmem_ld16(tq + L::TM_AO + NS * s2 + 16 * q, y);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = fmaf(dq, x[j], y[j]);
                if (t < ch.len) {
                    dst[2 * q] = bf16x8(x);
                    dst[2 * q + 1] = bf16x8(x + 8);
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_OD + s2]);
        }
    }

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
cudaError_t launch_chain(const Args& a, cudaStream_t s)
{
    using L = Cfg<D, NS>;
    CUtensorMap mq, mk, mv;
    if (!make_rows_map(&mq, a.q, a, a.Hk, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_rows_map(&mk, a.k, a, a.Hk, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_rows_map(&mv, a.v, a, a.H, NS, CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(chain_kernel<D, NS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)L::BYTES);
    if (e != cudaSuccess) return e;
    ChainArgs p{a, a.blk};
    ProfScope ps(kGdrChain, s);
    chain_kernel<D, NS><<<(unsigned)(chains(a) * (D / NS)), kThreads, L::BYTES, s>>>(mq, mk, mv, p);
    return cudaGetLastError();
}

}  // namespace

// Chain width.  (Figures: see the table in the header comment of launch_fwd_tc.)
cudaError_t launch_fwd_tc(const Args& a, cudaStream_t s)
{
    cudaError_t e = launch_operands_tc(a, s);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 148;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    if (a.D == 64) return launch_chain<64, 32>(a, s);
    return chains(a) * 4 <= sms ? launch_chain<128, 32>(a, s) : launch_chain<128, 64>(a, s);
}

}  // namespace gdr
}  // namespace mdn
