// The backward pass's forward sweep of the gated delta rule on sm_100a: one CTA per
// chain and NS of its d_v columns rebuilds the states from the saved Vtilde,
//     S <- aC S + K^T [gV_hi | gV_lo],     gV = Diag(gam) Vtilde,
// and, while it has each entering state in two bf16 terms, forms what needs it in
// full precision (the fp32 gate gradients):
//     A1 = K [S_hi | S_lo], Q [S_hi | S_lo]    (each M 64, N 2 NS, K 128)
//     XS = Diag(D) K S                     fp32, for the reverse chain's <XS, dv>
//     rows of scale Diag(D) (Q S) . dO     summed over the slice's columns
// The products of the update do not depend on the state, so nothing but the fp32
// update itself is sequential: the updates' products run ahead, and the entering
// states' tile and every TMEM result are double-buffered.  Bound by issue (the
// epilogues) and, for the outputs, by L2: per chunk and head 64 KB of fp32 states
// (for <G, S>), 32 KB of bf16 states (for the token gradients) and 32 KB of XS.
// 32 heads of 2048 tokens: 46 us, 1.4 us a chunk.
//
// Warps: 0 MMA issue, 1 loads, 16 chain warps (the state, K S and Q S as in the forward
// chain), 4 warps that form gV, 1 that stores the bf16 states (TMA from a tile of their
// own: 16-byte pieces from the chain warps, 32 rows an instruction, held them up).
#include "gdr_tc.cuh"

namespace mdn {
namespace gdr {
namespace {

using namespace sm100;
using namespace tc;
using inter::wait_bar;
using inter::warp_wait;

constexpr int D = 128;
constexpr int kChainWarp0 = 2, CW = 16, kAuxWarp0 = kChainWarp0 + CW, AW = 4;
constexpr int kStoreWarp = kAuxWarp0 + AW, kThreads = (kStoreWarp + 1) * 32;

template <int NS>
struct Cfg {
    static constexpr int NH = NS / 4;
    static constexpr int NV = NS == 32 ? 4 : 2;              // slots of Vtilde, dO and the record
    static constexpr int NK = NS == 32 ? 3 : 2;              // slots of K, Q
    static constexpr uint32_t KQ0 = 0;                       // [K; Q], NK slots
    static constexpr uint32_t ST0 = NK * 32768;              // [S_hi | S_lo], 2 slots
    static constexpr uint32_t ST_BYTES = D * 2 * NS * 2;
    static constexpr uint32_t SI = ST0 + 2 * ST_BYTES;       // the entering state in bf16, to be stored
    static constexpr uint32_t GV0 = SI + D * NS * 2;         // [gV_hi | gV_lo], 2 slots
    static constexpr uint32_t GV_BYTES = 64 * 2 * NS * 2;
    static constexpr uint32_t V_BYTES = 64 * NS * 2;
    static constexpr uint32_t V0 = GV0 + 2 * GV_BYTES;       // Vtilde slice, NV slots
    static constexpr uint32_t O0 = V0 + NV * V_BYTES;        // dO slice, NV slots
    static constexpr uint32_t CR0 = O0 + NV * V_BYTES;       // records
    static constexpr uint32_t BARS = CR0 + NV * kBwdRecBytes;
    static constexpr uint32_t MISC = BARS + 256;
    static constexpr uint32_t BYTES = MISC + 16;
    static_assert(BYTES <= 232448, "shared memory");
    static constexpr uint32_t TM_A1 = 0;        // K S, then Q S: 2 NS each
    static constexpr uint32_t TM_A2 = 4 * NS;   // 2 slots x 2 NS
    static constexpr uint32_t kTmemCols = 8 * NS;
    __device__ static __forceinline__ uint32_t off(int i, int c, int lo, uint32_t panel) {
        return NS == 32 ? sw128_off(i, 4 * lo + c) : lo * panel + sw128_off(i, c);
    }
    __device__ static __forceinline__ uint32_t v_off(int r, int c) {
        return NS == 32 ? sw64_off(r, c) : sw128_off(r, c);
    }
};

constexpr int B_FKQ = 0;   // [3] K, Q landed
constexpr int B_FVD = 3;   // [4] Vtilde, dO, record landed
constexpr int B_EVD = 7;   // [4] ... read
constexpr int B_M1 = 11;   // [2] A1 complete
constexpr int B_M2 = 13;   // [2] A2 complete (and the A1 before it)
constexpr int B_GV = 15;   // [2] gV written
constexpr int B_SR = 17;   // [2] next state written
constexpr int B_OD = 19;   //     A1 read
constexpr int B_SF = 20;   //     the bf16 state's tile has been stored
constexpr int B_KF = 21;   // [3] K, Q slot free (A1 complete, and the A2 before it)
constexpr int B_FIN = 24;
constexpr int kBars = 25;

template <int NS>
__global__ void __launch_bounds__(kThreads, 1)
rebuild_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_vt, const __grid_constant__ CUtensorMap tm_do,
               const __grid_constant__ CUtensorMap tm_sb, const Args a)
{
    using L = Cfg<NS>;
    constexpr int NH = L::NH, NP = NH / 8, SL = D / NS, NV = L::NV, NK = L::NK;
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
            if (k >= B_EVD && k < B_EVD + NV) count = CW + AW;
            if (k >= B_GV && k < B_GV + 2) count = AW;
            if (k >= B_SR && k <= B_OD) count = CW;
            mbar_init(&bars[k], count);
        }
        mbar_fence_init();
        *abort_flag = 0;
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, L::kTmemCols);
        tmem_relinquish();
    }
    const bool chain = warp >= kChainWarp0 && warp < kAuxWarp0;
    const int hc = (warp - kChainWarp0) >> 2;
    const int irow = quad * 32 + lid;
    float s[NH];
    // the state as the B operand (slot), and as the entering state of chunk n
    auto put_state = [&](int slot) {
#pragma unroll
        for (int c = 0; c < NP; ++c) {
            uint4 hi, lo;
            split8(s + 8 * c, hi, lo);
            const int cc = hc * NP + c;
            *reinterpret_cast<uint4*>(sm + L::ST0 + slot * L::ST_BYTES + L::off(irow, cc, 0, D * 128)) = hi;
            *reinterpret_cast<uint4*>(sm + L::ST0 + slot * L::ST_BYTES + L::off(irow, cc, 1, D * 128)) = lo;
            *reinterpret_cast<uint4*>(sm + L::SI + L::v_off(irow, cc)) = hi;
        }
    };
    auto store_state = [&](int n) {  // fp32, in the order these threads hold it
        float* dst = a.ssf + ((head_chunk(n) * SL + slice) * CW + (warp - kChainWarp0)) * (NH * 32) + 4 * lid;
#pragma unroll
        for (int j = 0; j < NH; j += 4)
            *reinterpret_cast<float4*>(dst + 32 * j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
    };
    const size_t srow0 = ((size_t)ch.state * D + irow) * D + j0 + NH * hc;
    if (chain) {
#pragma unroll
        for (int j = 0; j < NH; j += 4) {
            const float4 x = a.S0 ? *reinterpret_cast<const float4*>(a.S0 + srow0 + j)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            s[j] = x.x; s[j + 1] = x.y; s[j + 2] = x.z; s[j + 3] = x.w;
        }
        put_state(0);
        fence_proxy_async_smem();
        if (NT > 0) store_state(0);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tq = tmem + (static_cast<uint32_t>(quad * 32) << 16);

    if (warp == 0) {
        // ------------------------------------------------------------ MMA issue
        const uint64_t d_k0 = smem_desc(sbase + L::KQ0, 16, 1024, kSw128);
        const uint64_t d_kt0 = smem_desc(sbase + L::KQ0, 16384, 1024, kSw128);  // MN-major
        const uint64_t d_st0 = smem_desc(sbase + L::ST0, D * 128, 1024, kSw128);
        const uint64_t d_gv0 = smem_desc(sbase + L::GV0, 8192, 1024, kSw128);
        constexpr uint32_t id1 = idesc_bf16(64, 2 * NS, false, true);
        constexpr uint32_t id2 = idesc_bf16(128, 2 * NS, true, true);
        auto update = [&](int n) {  // A2 of chunk n; its TMEM slot was read before SR of n - 2
            const int s2 = n & 1, sk = n % NK;
            if (!warp_wait(&bars[B_FKQ + sk], (n / NK) & 1, abort_flag)) return false;
            if (!warp_wait(&bars[B_GV + s2], (n >> 1) & 1, abort_flag)) return false;
            tc_fence_after_sync();
            const uint64_t dkt = d_kt0 + sk * (32768 >> 4), dgv = d_gv0 + s2 * (L::GV_BYTES >> 4);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_bf16_elect(tmem + L::TM_A2 + 2 * NS * s2, dkt + ks * (2048 >> 4), dgv + ks * (2048 >> 4),
                               id2, ks > 0);
            mma_commit_elect(&bars[B_M2 + s2]);
            return true;
        };
        bool go = NT > 0 && update(0);
        for (int n = 0; n < NT && go; ++n) {
            const int s2 = n & 1;
            if (n >= 1 && !warp_wait(&bars[B_SR + (s2 ^ 1)], ((n - 1) >> 1) & 1, abort_flag)) break;
            if (n >= 1 && !warp_wait(&bars[B_OD], (n - 1) & 1, abort_flag)) break;
            tc_fence_after_sync();
            const uint64_t dk = d_k0 + (n % NK) * (32768 >> 4), dst = d_st0 + s2 * (L::ST_BYTES >> 4);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const uint64_t d = dk + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4);
                mma_bf16_elect(tmem + L::TM_A1, d, dst + ks * (2048 >> 4), id1, ks > 0);
                mma_bf16_elect(tmem + L::TM_A1 + 2 * NS, d + (8192 >> 4), dst + ks * (2048 >> 4), id1, ks > 0);
            }
            mma_commit_elect(&bars[B_M1 + s2]);
            mma_commit_elect(&bars[B_KF + n % NK]);
            // the next update needs no state; the state it follows is one epilogue away
            if (n + 1 < NT && !update(n + 1)) break;
        }
        mma_commit_elect(&bars[B_FIN]);
        (void)mbar_wait(&bars[B_FIN], 0);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ loads
        if (lid == 0) {
            int done_kq = 0, done_vd = 0;
            for (int n = 0; n < NT; ++n) {
                const int sk = n % NK, sv = n % NV, t = tt0 + n * kChunk;
                if (n >= NV && !wait_bar(&bars[B_EVD + sv], ((n / NV) - 1) & 1, abort_flag)) break;
                uint64_t* fb = &bars[B_FVD + sv];
                mbar_arrive_expect_tx(fb, 2 * L::V_BYTES + kBwdRecBytes);
                tma_load_4d(sm + L::V0 + sv * L::V_BYTES, &tm_vt, j0, ch.h, t, tb, fb);
                tma_load_4d(sm + L::O0 + sv * L::V_BYTES, &tm_do, j0, ch.h, t, tb, fb);
                bulk_load(sm + L::CR0 + sv * kBwdRecBytes, a.blk + head_chunk(n) * kBwdBytes + kBwdImg,
                          kBwdRecBytes, fb);
                done_vd = n + 1;
                if (n >= NK && !wait_bar(&bars[B_KF + sk], ((n / NK) - 1) & 1, abort_flag)) break;
                fb = &bars[B_FKQ + sk];
                mbar_arrive_expect_tx(fb, 32768);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint8_t* dst = sm + L::KQ0 + sk * 32768 + q * 16384;
                    tma_load_4d(dst, &tm_k, q * 64, ch.hk, t, tb, fb);
                    tma_load_4d(dst + 8192, &tm_q, q * 64, ch.hk, t, tb, fb);
                }
                done_kq = n + 1;
            }
            for (int n = done_kq - NK; n < done_kq; ++n)
                if (n >= 0) (void)mbar_wait(&bars[B_FKQ + n % NK], (n / NK) & 1);
            for (int n = done_vd - NV; n < done_vd; ++n)
                if (n >= 0) (void)mbar_wait(&bars[B_FVD + n % NV], (n / NV) & 1);
        }
        __syncwarp();
    } else if (chain) {
        // ------------------------------------------------------------ the state, and A1's epilogue
        const int r0 = quad * 16 + (lid >> 2), pc = (lid & 3) * 4;
        for (int n = 0; n < NT; ++n) {
            const int s2 = n & 1, sv = n % NV;
            if (!warp_wait(&bars[B_FVD + sv], (n / NV) & 1, abort_flag)) break;
            const float* cr = reinterpret_cast<const float*>(sm + L::CR0 + sv * kBwdRecBytes);
            const float aC = cr[kRecBwdB];
            const float dr[2] = {cr[kRecD + r0], cr[kRecD + r0 + 8]}, dq[2] = {cr[kRecDq + r0], cr[kRecDq + r0 + 8]};
            uint32_t ow[NP][2];
#pragma unroll
            for (int c = 0; c < NP; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    ow[c][e] = *reinterpret_cast<const uint32_t*>(sm + L::O0 + sv * L::V_BYTES +
                                                                  L::v_off(r0 + 8 * e, hc * NP + c) + pc);
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_EVD + sv]);
            if (!warp_wait(&bars[B_M2 + s2], (n >> 1) & 1, abort_flag)) break;
            tc_fence_after_sync();
            {
                float u[NH], w[NH];
                if constexpr (NH == 8) {
                    tmem_ld8(tq + L::TM_A2 + 2 * NS * s2 + NH * hc, u);
                    tmem_ld8(tq + L::TM_A2 + 2 * NS * s2 + NS + NH * hc, w);
                } else {
                    tmem_ld16(tq + L::TM_A2 + 2 * NS * s2 + NH * hc, u);
                    tmem_ld16(tq + L::TM_A2 + 2 * NS * s2 + NS + NH * hc, w);
                }
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < NH; ++j) s[j] = fmaf(aC, s[j], u[j] + w[j]);
            }
            // the other slot's reader, A1 of chunk n - 1, was waited for below; the tile of
            // the bf16 state has been stored
            if (n + 1 < NT) {
                if (!warp_wait(&bars[B_SF], n & 1, abort_flag)) break;
                put_state(s2 ^ 1);
            }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_SR + s2]);
            if (n + 1 < NT) store_state(n + 1);
            if (!warp_wait(&bars[B_M1 + s2], (n >> 1) & 1, abort_flag)) break;
            tc_fence_after_sync();
            float x[NP * 4], y[NP * 4], u[NP * 4], w[NP * 4];
            tmem_ld_16x256<NP>(tq + L::TM_A1 + NH * hc, x);
            tmem_ld_16x256<NP>(tq + L::TM_A1 + NS + NH * hc, y);
            tmem_ld_16x256<NP>(tq + L::TM_A1 + 2 * NS + NH * hc, u);
            tmem_ld_16x256<NP>(tq + L::TM_A1 + 3 * NS + NH * hc, w);
            tmem_wait_ld();
            tc_fence_before_sync();
            __syncwarp();
            if (lid == 0) mbar_arrive(&bars[B_OD]);
            float po[2] = {0.f, 0.f};
            float* xs = a.xs + ((head_chunk(n) * SL + slice) * CW + (warp - kChainWarp0)) * (NP * 128) + 4 * lid;
#pragma unroll
            for (int c = 0; c < NP; ++c) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 4 * c + 2 * e;
                    float o0, o1;
                    unpack2(ow[c][e], o0, o1);
                    po[e] = fmaf(u[i] + w[i], o0, fmaf(u[i + 1] + w[i + 1], o1, po[e]));
                }
                *reinterpret_cast<float4*>(xs + 128 * c) =
                    make_float4(dr[0] * (x[4 * c] + y[4 * c]), dr[0] * (x[4 * c + 1] + y[4 * c + 1]),
                                dr[1] * (x[4 * c + 2] + y[4 * c + 2]), dr[1] * (x[4 * c + 3] + y[4 * c + 3]));
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                po[e] += __shfl_xor_sync(0xffffffffu, po[e], 1);
                po[e] += __shfl_xor_sync(0xffffffffu, po[e], 2);
                if ((lid & 3) == 0)
                    a.po[((head_chunk(n) * SL + slice) * 4 + hc) * kChunk + r0 + 8 * e] = dq[e] * po[e];
            }
        }
    } else if (warp == kStoreWarp) {
        // ------------------------------------------------------------ the bf16 states
        for (int n = 0; n < NT; ++n) {
            if (n >= 1 && !warp_wait(&bars[B_SR + ((n - 1) & 1)], ((n - 1) >> 1) & 1, abort_flag)) break;
            if (lid == 0) {
                tma_store_3d(&tm_sb, j0, 0, (int)head_chunk(n), sm + L::SI);
                bulk_commit_group();
                bulk_wait_group_read<0>();
                mbar_arrive(&bars[B_SF]);
            }
            __syncwarp();
        }
        if (lid == 0) bulk_wait_group_all();
    } else {
        // ------------------------------------------------------------ gV
        const int ot = tid - kAuxWarp0 * 32, r = ot >> 1, h0 = (ot & 1) * (NS / 16);  // half a row each
        for (int n = 0; n < NT; ++n) {
            const int s2 = n & 1, sv = n % NV, valid = ch.len - n * kChunk;
            if (!warp_wait(&bars[B_FVD + sv], (n / NV) & 1, abort_flag)) break;
            const float g = reinterpret_cast<const float*>(sm + L::CR0 + sv * kBwdRecBytes)[kRecGam + r];
            if (n >= 2 && !warp_wait(&bars[B_M2 + s2], ((n - 2) >> 1) & 1, abort_flag)) break;
#pragma unroll
            for (int c = 0; c < NS / 16; ++c) {
                float x[8];
                unpack_bf16x8(*reinterpret_cast<const uint4*>(sm + L::V0 + sv * L::V_BYTES + L::v_off(r, h0 + c)), x);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = r < valid ? g * x[e] : 0.f;
                uint4 hi, lo;
                split8(x, hi, lo);
                *reinterpret_cast<uint4*>(sm + L::GV0 + s2 * L::GV_BYTES + L::off(r, h0 + c, 0, 8192)) = hi;
                *reinterpret_cast<uint4*>(sm + L::GV0 + s2 * L::GV_BYTES + L::off(r, h0 + c, 1, 8192)) = lo;
            }
            if (valid < kChunk && a.cu_s) {
                // K rows behind the sequence may hold anything: zeros, as in the forward chain
                if (!warp_wait(&bars[B_FKQ + n % NK], (n / NK) & 1, abort_flag)) break;
                for (int e = ot; e < 64 * 16; e += AW * 32) {
                    const int rr = e >> 4, q = e & 15;
                    if (rr >= valid)
                        *reinterpret_cast<uint4*>(sm + L::KQ0 + (n % NK) * 32768 + (q >> 3) * 16384 + sw128_off(rr, q & 7)) =
                            make_uint4(0, 0, 0, 0);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lid == 0) {
                mbar_arrive(&bars[B_GV + s2]);
                mbar_arrive(&bars[B_EVD + sv]);
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (*abort_flag && tid == 0) atomicOr(a.status + 1, 1u);
    if (warp == 0) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

template <int NS>
cudaError_t launch_typed(const Args& a, cudaStream_t s)
{
    using L = Cfg<NS>;
    CUtensorMap mq, mk, mv, mo, ms;
    const auto sw = NS == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    if (!make_rows_map(&mq, a.q, a, a.Hk, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_rows_map(&mk, a.k, a, a.Hk, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_rows_map(&mv, a.vt, a, a.H, NS, sw) || !make_rows_map(&mo, a.d_o, a, a.H, NS, sw) ||
        !make_states_map(&ms, a.sb, a, NS, sw))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(rebuild_kernel<NS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)L::BYTES);
    if (e != cudaSuccess) return e;
    ProfScope ps(kGdrBwdStates, s);
    rebuild_kernel<NS><<<(unsigned)(chains(a) * (D / NS)), kThreads, L::BYTES, s>>>(mq, mk, mv, mo, ms, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rebuild_tc(const Args& a, int ns, cudaStream_t s)
{
    return ns == 32 ? launch_typed<32>(a, s) : launch_typed<64>(a, s);
}

}  // namespace gdr
}  // namespace mdn
