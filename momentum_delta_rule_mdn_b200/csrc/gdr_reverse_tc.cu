// The backward pass's reverse chain of the gated delta rule on sm_100a (formulas in
// gdr_tc.cuh): one CTA per chain and NS of its d_v columns, walking the chunks
// backwards with the adjoint G of the state in fp32 registers.  It has the shape of
// the forward chain, three dependent rounds per chunk and two products beside them:
//   R  = (Att'_hi + Att'_lo)^T dO                      (M 64, N NS, K 64)
//   A1 = K [G_hi | G_lo]                               (M 64, N 2 NS, K 128)
//   E' = R + Diag(gamU) K G, as two bf16 terms
//   AT = (T'_hi + T'_lo)^T [E'_hi | E'_lo]             (M 64, N 2 NS, K 64)
//   E  = AT_hi + AT_lo,  dv = beta E,  then -Diag(D) dv as two bf16 terms
//   A2 = Q^T [DqdO_hi | DqdO_lo] + K^T [-Ddv_hi | -Ddv_lo]   (M 128, N 2 NS, K 64)
//   G <- aC G + A2
// (T'^T and Att'^T are the images read MN-major.)  R runs under the state's epilogue of
// the chunk before, the Q^T product under that of E'; the 4 output warps form
// Diag(Dq) dO and store dv.  While the chain warps wait for products they take what the
// gate gradients need: aC <G, S> with the state entering the chunk, vtilde . E (dbeta),
// XS . dv and gam_r (G^T k_r) . vtilde_r, summed over this CTA's columns; and they
// store G in bf16 for the token gradients.  Bounds and hand-offs as in the forward chain; 32 heads of 2048 tokens:
// 75 us, 2.3 us a chunk (the forward chain's 1.65, two products and the gates' rows more).
#include "gdr_tc.cuh"

namespace mdn {
namespace gdr {
namespace {

using namespace sm100;
using namespace tc;
using inter::wait_bar;
using inter::warp_wait;

constexpr int D = 128;
constexpr int kChainWarp0 = 2, CW = 16, kOutWarp0 = kChainWarp0 + CW, OW = 4;
constexpr int kStoreWarp = kOutWarp0 + OW, kThreads = (kStoreWarp + 1) * 32;
constexpr int NV = 2;  // slots of Vtilde, dO, the record

template <int NS>
struct Cfg {
    static constexpr int NH = NS / 4;
    static constexpr int NFB = NS == 32 ? 2 : 1;              // slots of the images
    static constexpr uint32_t KQ0 = 0;                        // [K; Q], 2 slots
    static constexpr uint32_t FB0 = 2 * 32768;                // T'_hi, Att'_hi, T'_lo, Att'_lo
    static constexpr uint32_t ST = FB0 + NFB * kBwdImg;       // [G_hi | G_lo]
    // G in bf16, to be stored by TMA (64 columns: no room, the chain warps store it)
    static constexpr bool kTile = NS == 32;
    static constexpr uint32_t GI = ST + D * 2 * NS * 2;
    static constexpr uint32_t YB = GI + (kTile ? D * NS * 2 : 0);  // E' terms, then -D dv terms
    static constexpr uint32_t V_BYTES = 64 * NS * 2;
    static constexpr uint32_t EO = YB + 2 * V_BYTES;          // Dq dO terms
    static constexpr int NEO = NS == 32 ? 2 : 1;              // its slots
    static constexpr uint32_t VB = EO + NEO * 2 * V_BYTES;    // bf16 dv and its rest
    static constexpr uint32_t VL = VB + V_BYTES;
    static constexpr uint32_t V0 = VL + V_BYTES;              // Vtilde, NV slots
    static constexpr uint32_t O0 = V0 + NV * V_BYTES;         // dO, NV slots (an operand of R)
    static constexpr uint32_t CR0 = O0 + NV * V_BYTES;        // records
    static constexpr uint32_t BARS = CR0 + NV * kBwdRecBytes;
    static constexpr uint32_t MISC = BARS + 256;
    static constexpr uint32_t BYTES = MISC + 16;
    static_assert(BYTES <= 232448, "shared memory");
    static constexpr uint32_t TM_KG = 0;         // 2 NS
    static constexpr uint32_t TM_AT = 2 * NS;    // 2 NS
    static constexpr uint32_t TM_A2 = 4 * NS;    // 2 NS
    static constexpr uint32_t TM_R = 6 * NS;     // 2 slots x NS
    static constexpr uint32_t kTmemCols = 8 * NS;
    __device__ static __forceinline__ uint32_t off(int i, int c, int lo, uint32_t panel) {
        return NS == 32 ? sw128_off(i, 4 * lo + c) : lo * panel + sw128_off(i, c);
    }
    __device__ static __forceinline__ uint32_t v_off(int r, int c) {
        return NS == 32 ? sw64_off(r, c) : sw128_off(r, c);
    }
};

constexpr int B_FKQ = 0;   // [2] K, Q landed
constexpr int B_FFB = 2;   // [2] images landed
constexpr int B_FVD = 4;   // [NV] Vtilde, dO, record landed
constexpr int B_EVD = 6;   // [NV] ... read (after A1 of the chunk, so after R)
constexpr int B_M1 = 8;    //     A1 (and R) complete
constexpr int B_MT = 9;    // [2] AT complete (the images' slot is free)
constexpr int B_M2 = 11;   // [2] A2 complete (the K, Q slot is free)
constexpr int B_YR = 13;   //     E' written
constexpr int B_GR = 14;   //     -D dv written
constexpr int B_VR = 15;   //     dv tiles written
constexpr int B_SR = 16;   //     next adjoint written
constexpr int B_EO = 17;   // [2] Dq dO written, rows behind the sequence cleared (two: the first two
                           //     chunks' are formed with nothing waited for in between)
constexpr int B_VF = 19;   //     dv tiles stored
constexpr int B_GF = 20;   //     the bf16 adjoint's tile has been stored
constexpr int B_FIN = 21;
constexpr int kBars = 22;

template <int NS>
__global__ void __launch_bounds__(kThreads, 1)
reverse_kernel_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_vt, const __grid_constant__ CUtensorMap tm_do,
                  const __grid_constant__ CUtensorMap tm_dv, const __grid_constant__ CUtensorMap tm_dvl,
                  const __grid_constant__ CUtensorMap tm_gb,
                  const Args a)
{
    using L = Cfg<NS>;
    constexpr int NH = L::NH, NP = NH / 8, SL = D / NS;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, lid = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int quad = warp & 3, slice = blockIdx.x % SL, j0 = slice * NS;
    const Chain ch = chain_of(a, blockIdx.x / SL);
    const int NT = (ch.len + kChunk - 1) / kChunk;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BARS);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC + 4);
    const int tb = a.cu_s ? 0 : (int)(ch.row0 / (a.T > 0 ? a.T : 1));
    const int tt0 = a.cu_s ? (int)ch.row0 : 0;
    auto head_chunk = [&](int n) { return (size_t)(ch.chunk0 + n) * a.H + ch.h; };

    if (tid == 0) {
        for (int k = 0; k < kBars; ++k) {
            uint32_t count = 1;
            if (k >= B_EVD && k < B_EVD + NV) count = CW + OW;
            if (k >= B_YR && k <= B_SR) count = CW;
            if (k >= B_EO && k <= B_VF) count = OW;
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
    const int hc = (warp - kChainWarp0) >> 2;
    const int irow = quad * 32 + lid;
    float g[NH];
    auto put_state = [&]() {
#pragma unroll
        for (int c = 0; c < NP; ++c) {
            uint4 hi, lo;
            split8(g + 8 * c, hi, lo);
            const int cc = hc * NP + c;
            *reinterpret_cast<uint4*>(sm + L::ST + L::off(irow, cc, 0, D * 128)) = hi;
            *reinterpret_cast<uint4*>(sm + L::ST + L::off(irow, cc, 1, D * 128)) = lo;
            if (L::kTile) *reinterpret_cast<uint4*>(sm + L::GI + L::v_off(irow, cc)) = hi;
        }
    };
    const size_t srow0 = ((size_t)ch.state * D + irow) * D + j0 + NH * hc;
    if (chain) {
#pragma unroll
        for (int j = 0; j < NH; j += 4) {
            const float4 x = a.dS_T ? *reinterpret_cast<const float4*>(a.dS_T + srow0 + j)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
            g[j] = x.x; g[j + 1] = x.y; g[j + 2] = x.z; g[j + 3] = x.w;
        }
        put_state();
        fence_proxy_async_smem();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tq = tmem + (static_cast<uint32_t>(quad * 32) << 16);

    // m counts the chunks processed: chunk n = NT - 1 - m
    if (warp == 0) {
        // ------------------------------------------------------------ MMA issue
        const uint64_t d_k0 = smem_desc(sbase + L::KQ0, 16, 1024, kSw128);
        const uint64_t d_kt0 = smem_desc(sbase + L::KQ0, 16384, 1024, kSw128);         // K^T
        const uint64_t d_qt0 = smem_desc(sbase + L::KQ0 + 8192, 16384, 1024, kSw128);  // Q^T
        const uint64_t d_st = smem_desc(sbase + L::ST, D * 128, 1024, kSw128);
        const uint64_t d_fb0 = smem_desc(sbase + L::FB0, 8192, 1024, kSw128);          // MN-major
        const uint64_t d_y = smem_desc(sbase + L::YB, 8192, 1024, kSw128);
        const uint64_t d_eo = smem_desc(sbase + L::EO, 8192, 1024, kSw128);
        const uint64_t d_o0 = NS == 32 ? smem_desc(sbase + L::O0, 4096, 512, kSw64)
                                       : smem_desc(sbase + L::O0, 8192, 1024, kSw128);
        constexpr uint32_t ostep = (16 * NS * 2) >> 4;
        constexpr uint32_t id1 = idesc_bf16(64, 2 * NS, false, true);
        constexpr uint32_t idt = idesc_bf16(64, 2 * NS, true, true);
        constexpr uint32_t idr = idesc_bf16(64, NS, true, true);
        constexpr uint32_t id2 = idesc_bf16(128, 2 * NS, true, true);
        auto rpart = [&](int m) {  // R of chunk m; its slot was read before SR of m - 2
            const int sf = m % L::NFB, sv = m % NV;
            if (!warp_wait(&bars[B_FFB + sf], (m / L::NFB) & 1, abort_flag)) return false;
            if (!warp_wait(&bars[B_EO + (m & 1)], (m >> 1) & 1, abort_flag)) return false;
            tc_fence_after_sync();
            const uint64_t df = d_fb0 + sf * (kBwdImg >> 4), dO_ = d_o0 + sv * (L::V_BYTES >> 4);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_bf16_elect(tmem + L::TM_R + NS * (m & 1), df + (kBlkAtt >> 4) + ks * (2048 >> 4),
                               dO_ + ks * ostep, idr, ks > 0);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_bf16_elect(tmem + L::TM_R + NS * (m & 1), df + (kBwdAttLo >> 4) + ks * (2048 >> 4),
                               dO_ + ks * ostep, idr, 1);
            return true;
        };
        bool go = NT > 0 && warp_wait(&bars[B_FKQ], 0, abort_flag) && rpart(0);
        for (int m = 0; m < NT && go; ++m) {
            const int s2 = m & 1, sf = m % L::NFB;
            if (m >= 1 && !warp_wait(&bars[B_SR], (m - 1) & 1, abort_flag)) break;
            tc_fence_after_sync();
            const uint64_t dk = d_k0 + s2 * (32768 >> 4), df = d_fb0 + sf * (kBwdImg >> 4);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
                mma_bf16_elect(tmem + L::TM_KG, dk + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4),
                               d_st + ks * (2048 >> 4), id1, ks > 0);
            mma_commit_elect(&bars[B_M1]);
            // under the E' epilogue: Q^T Diag(Dq) dO
            const uint64_t deo = d_eo + (m % L::NEO) * ((2 * L::V_BYTES) >> 4);
            const uint64_t dqt = d_qt0 + s2 * (32768 >> 4), dkt = d_kt0 + s2 * (32768 >> 4);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_bf16_elect(tmem + L::TM_A2, dqt + ks * (2048 >> 4), deo + ks * (2048 >> 4), id2, ks > 0);
            if (!warp_wait(&bars[B_YR], m & 1, abort_flag)) break;
            tc_fence_after_sync();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_bf16_elect(tmem + L::TM_AT, df + ks * (2048 >> 4), d_y + ks * (2048 >> 4), idt, ks > 0);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_bf16_elect(tmem + L::TM_AT, df + (kBlkTlo >> 4) + ks * (2048 >> 4), d_y + ks * (2048 >> 4), idt, 1);
            mma_commit_elect(&bars[B_MT + s2]);
            if (m + 1 < NT && !warp_wait(&bars[B_FKQ + ((m + 1) & 1)], ((m + 1) >> 1) & 1, abort_flag)) break;
            if (!warp_wait(&bars[B_GR], m & 1, abort_flag)) break;
            tc_fence_after_sync();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_bf16_elect(tmem + L::TM_A2, dkt + ks * (2048 >> 4), d_y + ks * (2048 >> 4), id2, 1);
            mma_commit_elect(&bars[B_M2 + s2]);
            // under the state's epilogue: R of the next chunk (under that of dv its images' load is
            // still waited for, and the wait holds up A2)
            if (m + 1 < NT && !rpart(m + 1)) break;
        }
        mma_commit_elect(&bars[B_FIN]);
        (void)mbar_wait(&bars[B_FIN], 0);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ loads
        if (lid == 0) {
            int done_kq = 0, done_fb = 0, done_vd = 0;
            for (int m = 0; m < NT; ++m) {
                const int n = NT - 1 - m, s2 = m & 1, sv = m % NV, sf = m % L::NFB, t = tt0 + n * kChunk;
                const uint8_t* blk = a.blk + head_chunk(n) * kBwdBytes;
                // the images first: their slot is free before the K, Q slot is
                if (m >= L::NFB && !wait_bar(&bars[B_MT + ((m - L::NFB) & 1)], ((m - L::NFB) >> 1) & 1, abort_flag)) break;
                uint64_t* fb = &bars[B_FFB + sf];
                mbar_arrive_expect_tx(fb, kBwdImg);
                bulk_load(sm + L::FB0 + sf * kBwdImg, blk, kBwdImg, fb);
                done_fb = m + 1;
                if (m >= NV && !wait_bar(&bars[B_EVD + sv], ((m / NV) - 1) & 1, abort_flag)) break;
                fb = &bars[B_FVD + sv];
                mbar_arrive_expect_tx(fb, 2 * L::V_BYTES + kBwdRecBytes);
                tma_load_4d(sm + L::V0 + sv * L::V_BYTES, &tm_vt, j0, ch.h, t, tb, fb);
                tma_load_4d(sm + L::O0 + sv * L::V_BYTES, &tm_do, j0, ch.h, t, tb, fb);
                bulk_load(sm + L::CR0 + sv * kBwdRecBytes, blk + kBwdImg, kBwdRecBytes, fb);
                done_vd = m + 1;
                if (m >= 2 && !wait_bar(&bars[B_M2 + s2], ((m - 2) >> 1) & 1, abort_flag)) break;
                fb = &bars[B_FKQ + s2];
                mbar_arrive_expect_tx(fb, 32768);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint8_t* dst = sm + L::KQ0 + s2 * 32768 + q * 16384;
                    tma_load_4d(dst, &tm_k, q * 64, ch.hk, t, tb, fb);
                    tma_load_4d(dst + 8192, &tm_q, q * 64, ch.hk, t, tb, fb);
                }
                done_kq = m + 1;
            }
            for (int m = done_kq - 2; m < done_kq; ++m)
                if (m >= 0) (void)mbar_wait(&bars[B_FKQ + (m & 1)], (m >> 1) & 1);
            for (int m = done_fb - L::NFB; m < done_fb; ++m)
                if (m >= 0) (void)mbar_wait(&bars[B_FFB + m % L::NFB], (m / L::NFB) & 1);
            for (int m = done_vd - NV; m < done_vd; ++m)
                if (m >= 0) (void)mbar_wait(&bars[B_FVD + m % NV], (m / NV) & 1);
        }
        __syncwarp();
    } else if (chain) {
        // ------------------------------------------------------------ chain epilogues
        const int r0 = quad * 16 + (lid >> 2), pc = (lid & 3) * 4;
        // XS of this thread's rows and columns, and its part of the state entering the chunk:
        // loaded a chunk ahead, where they are used
        float4 xs[NP], se[NH / 4];
        auto load_xs = [&](int n) {
#pragma unroll
            for (int c = 0; c < NP; ++c)
                xs[c] = *reinterpret_cast<const float4*>(
                    a.xs + ((head_chunk(n) * SL + slice) * CW + (warp - kChainWarp0)) * (NP * 128) + 128 * c + 4 * lid);
        };
        auto load_se = [&](int n) {
            const float* src = a.ssf + ((head_chunk(n) * SL + slice) * CW + (warp - kChainWarp0)) * (NH * 32) + 4 * lid;
#pragma unroll
            for (int j = 0; j < NH / 4; ++j) se[j] = *reinterpret_cast<const float4*>(src + 128 * j);
        };
        if (NT > 0) {
            load_xs(NT - 1);
            load_se(NT - 1);
        }
        for (int m = 0; m < NT; ++m) {
            const int n = NT - 1 - m, s2 = m & 1, sv = m % NV, valid = ch.len - n * kChunk;
            const size_t hcn = head_chunk(n);
            if (!warp_wait(&bars[B_FVD + sv], (m / NV) & 1, abort_flag)) break;
            const float* cr = reinterpret_cast<const float*>(sm + L::CR0 + sv * kBwdRecBytes);
            const float aC = cr[kRecBwdB];
            float gu[2], be[2], dd[2];
            uint32_t vw[NP][2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                gu[e] = cr[kRecGamU + r0 + 8 * e];
                be[e] = cr[kRecBeta + r0 + 8 * e];
                dd[e] = -be[e] * cr[kRecD + r0 + 8 * e];
#pragma unroll
                for (int c = 0; c < NP; ++c)
                    vw[c][e] = *reinterpret_cast<const uint32_t*>(sm + L::V0 + sv * L::V_BYTES +
                                                                  L::v_off(r0 + 8 * e, hc * NP + c) + pc);
            }
            if (!warp_wait(&bars[B_M1], m & 1, abort_flag)) break;
            tc_fence_after_sync();
            if (lid == 0) mbar_arrive(&bars[B_EVD + sv]);
            float x[NP * 4], y[NP * 4], z[NP * 4];
            tmem_ld_16x256<NP>(tq + L::TM_KG + NH * hc, x);
            tmem_ld_16x256<NP>(tq + L::TM_KG + NS + NH * hc, y);
            tmem_ld_16x256<NP>(tq + L::TM_R + NS * s2 + NH * hc, z);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < NP; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 4 * c + 2 * e, r = r0 + 8 * e, cc = hc * NP + c;
                    float v0 = fmaf(gu[e], x[i] + y[i], z[i]);
                    float v1 = fmaf(gu[e], x[i + 1] + y[i + 1], z[i + 1]);
                    if (r >= valid) v0 = v1 = 0.f;
                    uint32_t hi, lo;
                    split2(v0, v1, hi, lo);
                    *reinterpret_cast<uint32_t*>(sm + L::YB + L::off(r, cc, 0, 8192) + pc) = hi;
                    *reinterpret_cast<uint32_t*>(sm + L::YB + L::off(r, cc, 1, 8192) + pc) = lo;
                }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_YR]);
            // while AT runs: the gates' sums with G, and G for the token gradients
            {
                float pw[2] = {0.f, 0.f};
#pragma unroll
                for (int c = 0; c < NP; ++c)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int i = 4 * c + 2 * e;
                        float v0, v1;
                        unpack2(vw[c][e], v0, v1);
                        pw[e] = fmaf(v0, x[i] + y[i], fmaf(v1, x[i + 1] + y[i + 1], pw[e]));
                    }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    pw[e] += __shfl_xor_sync(0xffffffffu, pw[e], 1);
                    pw[e] += __shfl_xor_sync(0xffffffffu, pw[e], 2);
                    if ((lid & 3) == 0)
                        a.pw[((hcn * SL + slice) * 4 + hc) * kChunk + r0 + 8 * e] = gu[e] * be[e] * pw[e];
                }
                float t = 0.f;
#pragma unroll
                for (int j = 0; j < NH; j += 4)
                    t = fmaf(g[j], se[j / 4].x, fmaf(g[j + 1], se[j / 4].y,
                        fmaf(g[j + 2], se[j / 4].z, fmaf(g[j + 3], se[j / 4].w, t))));
                if (n > 0) load_se(n - 1);
#pragma unroll
                for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                if (lid == 0) a.gs[(hcn * SL + slice) * CW + (warp - kChainWarp0)] = aC * t;
                if (!L::kTile)
#pragma unroll
                    for (int c = 0; c < NP; ++c)
                        *reinterpret_cast<uint4*>(a.gb + (hcn * D + irow) * D + j0 + NH * hc + 8 * c) = bf16x8(g + 8 * c);
            }
            // the last chunk's dv has left
            if (m >= 1 && !warp_wait(&bars[B_VF], (m - 1) & 1, abort_flag)) break;
            if (!warp_wait(&bars[B_MT + s2], (m >> 1) & 1, abort_flag)) break;
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
                    split2(dd[e] * x[i], dd[e] * x[i + 1], hi, lo);
                    *reinterpret_cast<uint32_t*>(sm + L::YB + L::off(r, cc, 0, 8192) + pc) = hi;
                    *reinterpret_cast<uint32_t*>(sm + L::YB + L::off(r, cc, 1, 8192) + pc) = lo;
                }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_GR]);
            float pb[2] = {0.f, 0.f}, px[2] = {0.f, 0.f};
#pragma unroll
            for (int c = 0; c < NP; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 4 * c + 2 * e;
                    float v0, v1;
                    unpack2(vw[c][e], v0, v1);
                    pb[e] = fmaf(v0, x[i], fmaf(v1, x[i + 1], pb[e]));
                    const float d0 = be[e] * x[i], d1 = be[e] * x[i + 1];
                    px[e] = e ? fmaf(xs[c].z, d0, fmaf(xs[c].w, d1, px[e])) : fmaf(xs[c].x, d0, fmaf(xs[c].y, d1, px[e]));
                    uint32_t hi, lo;
                    split2(d0, d1, hi, lo);
                    const uint32_t at = L::v_off(r0 + 8 * e, hc * NP + c) + pc;
                    *reinterpret_cast<uint32_t*>(sm + L::VB + at) = hi;
                    *reinterpret_cast<uint32_t*>(sm + L::VL + at) = lo;
                }
            if (n > 0) load_xs(n - 1);
            fence_proxy_async_smem();
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_VR]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                pb[e] += __shfl_xor_sync(0xffffffffu, pb[e], 1);
                pb[e] += __shfl_xor_sync(0xffffffffu, pb[e], 2);
                px[e] += __shfl_xor_sync(0xffffffffu, px[e], 1);
                px[e] += __shfl_xor_sync(0xffffffffu, px[e], 2);
                if ((lid & 3) == 0) {
                    const size_t at = ((hcn * SL + slice) * 4 + hc) * kChunk + r0 + 8 * e;
                    a.pb[at] = pb[e];
                    a.px[at] = px[e];
                }
            }
            if (!warp_wait(&bars[B_M2 + s2], (m >> 1) & 1, abort_flag)) break;
            tc_fence_after_sync();
            {
                float u[NH], w[NH];
                if constexpr (NH == 8) {
                    tmem_ld8(tq + L::TM_A2 + NH * hc, u);
                    tmem_ld8(tq + L::TM_A2 + NS + NH * hc, w);
                } else {
                    tmem_ld16(tq + L::TM_A2 + NH * hc, u);
                    tmem_ld16(tq + L::TM_A2 + NS + NH * hc, w);
                }
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < NH; ++j) g[j] = fmaf(aC, g[j], u[j] + w[j]);
            }
            if (L::kTile && !warp_wait(&bars[B_GF], m & 1, abort_flag)) break;
            put_state();
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_SR]);
        }
    } else if (warp == kStoreWarp) {
        // ------------------------------------------------------------ G in bf16
        if (L::kTile) {
            for (int m = 0; m < NT; ++m) {
                if (m >= 1 && !warp_wait(&bars[B_SR], (m - 1) & 1, abort_flag)) break;
                if (lid == 0) {
                    tma_store_3d(&tm_gb, j0, 0, (int)head_chunk(NT - 1 - m), sm + L::GI);
                    bulk_commit_group();
                    bulk_wait_group_read<0>();
                    mbar_arrive(&bars[B_GF]);
                }
                __syncwarp();
            }
            if (lid == 0) bulk_wait_group_all();
        }
    } else {
        // ------------------------------------------------------------ Dq dO, and the stores of dv
        const int ot = tid - kOutWarp0 * 32, r = ot >> 1, h0 = (ot & 1) * (NS / 16), w0 = quad * 16;
        constexpr uint32_t kStrip = 16 * NS * 2;
        auto store_rows = [&](const uint8_t* tile, __nv_bfloat16* out, int n, int valid) {
            for (int e = lid; e < 16 * (NS / 8); e += 32) {
                const int rr = w0 + e / (NS / 8), c = e % (NS / 8);
                if (rr < valid)
                    *reinterpret_cast<uint4*>(out + ((size_t)(ch.row0 + n * kChunk + rr) * a.H + ch.h) * D + j0 + 8 * c) =
                        *reinterpret_cast<const uint4*>(tile + L::v_off(rr, c));
            }
        };
        auto form = [&](int m) {  // Diag(Dq) dO of chunk m; dO, K, Q rows behind the sequence become zero
            const int n = NT - 1 - m, s2 = m & 1, sv = m % NV, valid = ch.len - n * kChunk;
            if (!warp_wait(&bars[B_FVD + sv], (m / NV) & 1, abort_flag)) return false;
            const float q = reinterpret_cast<const float*>(sm + L::CR0 + sv * kBwdRecBytes)[kRecDq + r];
            // its tile was read by the Q^T product of chunk m - NEO (A2 complete)
            if (m >= L::NEO && !warp_wait(&bars[B_M2 + ((m - L::NEO) & 1)], ((m - L::NEO) >> 1) & 1, abort_flag)) return false;
            uint8_t* eo = sm + L::EO + (m % L::NEO) * 2 * L::V_BYTES;
#pragma unroll
            for (int c = 0; c < NS / 16; ++c) {
                uint8_t* src = sm + L::O0 + sv * L::V_BYTES + L::v_off(r, h0 + c);
                float x[8];
                unpack_bf16x8(*reinterpret_cast<const uint4*>(src), x);
                if (r >= valid) *reinterpret_cast<uint4*>(src) = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = r < valid ? q * x[e] : 0.f;
                uint4 hi, lo;
                split8(x, hi, lo);
                *reinterpret_cast<uint4*>(eo + L::off(r, h0 + c, 0, 8192)) = hi;
                *reinterpret_cast<uint4*>(eo + L::off(r, h0 + c, 1, 8192)) = lo;
            }
            if (valid < kChunk && a.cu_s) {
                if (!warp_wait(&bars[B_FKQ + s2], (m >> 1) & 1, abort_flag)) return false;
                for (int e = ot; e < 128 * 16; e += OW * 32) {
                    const int rr = e >> 4, p = e & 15;  // rows of K, then of Q
                    if ((rr & 63) >= valid)
                        *reinterpret_cast<uint4*>(sm + L::KQ0 + s2 * 32768 + (p >> 3) * 16384 + sw128_off(rr, p & 7)) =
                            make_uint4(0, 0, 0, 0);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lid == 0) {
                mbar_arrive(&bars[B_EO + s2]);
                mbar_arrive(&bars[B_EVD + sv]);
            }
            return true;
        };
        bool go = NT > 0 && form(0);
        for (int m = 0; m < NT && go; ++m) {
            const int n = NT - 1 - m;
            if (L::NEO == 2 && m + 1 < NT && !form(m + 1)) break;
            const int valid = min(kChunk, ch.len - n * kChunk);
            const bool whole = !a.cu_s || valid == kChunk;
            if (!warp_wait(&bars[B_VR], m & 1, abort_flag)) break;
            if (!whole) {
                store_rows(sm + L::VB, static_cast<__nv_bfloat16*>(a.dv), n, valid);
                store_rows(sm + L::VL, a.dvl, n, valid);
                __syncwarp();
            }
            if (lid == 0) {
                if (whole) {
                    tma_store_4d(&tm_dv, j0, ch.h, tt0 + n * kChunk + w0, tb, sm + L::VB + quad * kStrip);
                    tma_store_4d(&tm_dvl, j0, ch.h, tt0 + n * kChunk + w0, tb, sm + L::VL + quad * kStrip);
                    bulk_commit_group();
                }
                bulk_wait_group_read<0>();
                mbar_arrive(&bars[B_VF]);
            }
            __syncwarp();
            if (L::NEO == 1 && m + 1 < NT && !form(m + 1)) break;
        }
        if (lid == 0) bulk_wait_group_all();
    }

    tc_fence_before_sync();
    __syncthreads();
    const bool ok = *abort_flag == 0;
    if (chain && ok) {
#pragma unroll
        for (int j = 0; j < NH; j += 4)
            *reinterpret_cast<float4*>(a.dS0 + srow0 + j) = make_float4(g[j], g[j + 1], g[j + 2], g[j + 3]);
    }
    if (!ok && tid == 0) atomicOr(a.status + 1, 1u);
    if (warp == 0) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

template <int NS>
cudaError_t launch_typed(const Args& a, cudaStream_t s)
{
    using L = Cfg<NS>;
    CUtensorMap mq, mk, mv, mo, mdv, mdl, mg;
    const auto sw = NS == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    if (!make_rows_map(&mq, a.q, a, a.Hk, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_rows_map(&mk, a.k, a, a.Hk, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_rows_map(&mv, a.vt, a, a.H, NS, sw) || !make_rows_map(&mo, a.d_o, a, a.H, NS, sw) ||
        !make_rows_map(&mdv, a.dv, a, a.H, NS, sw, 16) || !make_rows_map(&mdl, a.dvl, a, a.H, NS, sw, 16) ||
        !make_states_map(&mg, a.gb, a, NS, sw))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(reverse_kernel_tc<NS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)L::BYTES);
    if (e != cudaSuccess) return e;
    ProfScope ps(kGdrBwdChain, s);
    reverse_kernel_tc<NS><<<(unsigned)(chains(a) * (D / NS)), kThreads, L::BYTES, s>>>(mq, mk, mv, mo, mdv, mdl, mg, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_reverse_tc(const Args& a, int ns, cudaStream_t s)
{
    return ns == 32 ? launch_typed<32>(a, s) : launch_typed<64>(a, s);
}

}  // namespace gdr
}  // namespace mdn
