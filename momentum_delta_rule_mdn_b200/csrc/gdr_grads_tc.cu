// The backward pass's token gradients of the gated delta rule on sm_100a: one CTA per
// chunk and key head, summing over the value heads that share it.  With L_{r,i} =
// exp(la_r - la_i), S the state entering the chunk and G the adjoint of the one leaving,
//     M1_{r,i} = scale L beta_i (do_r . vtilde_i)   (i <= r)
//     M2_{r,i} = L beta_i (dv_r . vtilde_i)         (i < r)
//     dq = Diag(Dq) dO S^T + M1 K
//     dk = Diag(gam) Vtilde G^T - Diag(D) dv S^T + M1^T Q - M2^T K - M2 K
// (all heads accumulate in the same two TMEM results), and for the gates
//     dbeta_r = vtilde_r . dv_r / beta_r                     (from the reverse chain)
// and dalpha_log_t as the sum of everything whose decay spans token t: with
// Z_{r,i} = M1_{r,i} q_r.k_i - M2_{r,i} k_r.k_i for i < r,
//     dalpha_log_t = aC <G, S> + sum_{r >= t} (scale D_r (S^T q_r) . do_r - XS_r . dv_r)
//                  + sum_{i < t} gam_i (G^T k_i) . vtilde_i + sum_{r >= t > i} Z_{r,i}.
// Every term of it carries the decay of token t.  The pairs are added up by blocks of 16 x 16:
// whole blocks behind and before t's, columns before t of the blocks behind, rows from t on of
// the blocks before, and t's rectangle of its diagonal block.  (The shorter recurrence
// dalpha_log_t = dalpha_log_{t+1} + q.dq - beta dbeta - ... adds and later takes off what
// each token does to itself: with alpha = e^-3 it lost 1.5e-4 of the result.  A suffix sum of
// Z's row sums less its column sums does so with the pairs behind t: a token of e^-8 among slow
// ones was 1e-3 off.)
//
// dq and dk are rounded to bf16, so S, G, M1, M2 and the scaled rows enter as single
// bf16 terms.  The gate gradients are fp32: their products P1, P2 and [K; Q] K^T have
// exact bf16 factors, dv in two terms.  P1 = dO Vtilde^T, P2 = dv Vtilde^T.
//
// One CTA per SM (176 KB of operands), walking the chunks; bound by the latency of its
// phases: [K; Q] K^T and the P products, the rows of M (twelve warps, a 32 x 16 block
// each) and the scaling of dO, Vtilde and dv in place, the products, the stores; the next
// chunk's loads run under the last.  A scheduler with one warp issues every fifth cycle at
// best, so the phases' work is spread over 16 warps.  32 heads of 2048 tokens: 65 us (one
// CTA a chunk took 73, on 8 warps 113).
#include "gdr_tc.cuh"

namespace mdn {
namespace gdr {
namespace {

using namespace sm100;
using namespace tc;
using inter::wait_bar;

constexpr int D = 128, kThreads = 512;
constexpr uint32_t KQ = 0;               // [K; Q]: 2 panels of 128 rows
constexpr uint32_t DV = 32768;           // [dv; dO]: the same
constexpr uint32_t VT = 65536;           // Vtilde: 2 panels of 64 rows
constexpr uint32_t DL = VT + 16384;      // dv's second term: the same (and 16 KB more are read behind it)
constexpr uint32_t SB = DL + 16384;      // S: 2 panels of 128 rows
constexpr uint32_t GB = SB + 32768;      // G
constexpr uint32_t M1 = GB + 32768;      // M1, -M2: 64 rows x 128 B
constexpr uint32_t M2 = M1 + 8192;
constexpr uint32_t VEC = M2 + 8192;      // gate vectors
constexpr uint32_t REC = VEC + 1024;     // the chunk's record
// Sums of Z by the warps that formed them, of M2's part and of M1's: [4 column blocks][128] of a
// block's rows (lanes 0..63 of M2, 64..127 of M1), [4 quads][2][64] of its columns, 16 rows each,
// [2][64] of the diagonal blocks' rectangles
constexpr uint32_t CS = REC + kBwdRecBytes;
constexpr int kCsCols = 512, kCsDiag = 1024;
constexpr uint32_t GS = CS + (1024 + 128) * 4;  // [4][64] sums of po, px, pb, pw over the slices; [256]: of gs
constexpr uint32_t BT = GS + 4 * 256 + 16;   // [4] block factors
constexpr uint32_t BARS = BT + 16;
constexpr uint32_t MISC = BARS + 48;
constexpr uint32_t BYTES = MISC + 16;
static_assert(BYTES <= 232448 && BARS % 8 == 0, "shared memory");
// TMEM: [K; Q] K^T 64, [P2; P1] 64, P2's second term 64, then dq 128, dk 128
constexpr uint32_t TM_G = 0, TM_P = 64, TM_PL = 128, TM_Q = 256, TM_K = 384;

struct GradMaps {
    CUtensorMap q, k, vt, d_o, dv, dvl, s, g, dq, dk;
};

__global__ void __launch_bounds__(kThreads, 1)
grads_kernel(const __grid_constant__ GradMaps tm, const Args a, const long long total)
{
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int quad = warp & 3;
    const int rep = a.H / a.Hk;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + BARS);  // [0] K, Q; [1] rows; [2] S, G; [3] P; [4] sums
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + MISC + 4);
    const int SL = D / a.ns;
    struct Item {
        long long n;
        int hk, tb, tt;
        ChunkRows cr;
    };
    auto item = [&](long long i) {  // valid <= 0 past the last chunk with tokens
        Item x;
        x.n = i / a.Hk;
        x.hk = (int)(i - x.n * a.Hk);
        x.cr.valid = 0;
        if (i < total) x.cr = chunk_rows(a, x.n);
        x.tb = a.cu_s ? 0 : (int)(x.n / a.NT);
        x.tt = a.cu_s ? (int)x.cr.row0 : (int)(x.n % a.NT) * kChunk;
        return x;
    };

    if (tid == 0) {
        for (int k = 0; k < 5; ++k) mbar_init(&bars[k], 1);
        mbar_fence_init();
        *abort_flag = 0;
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    for (int e = tid; e < 16384 / 16; e += kThreads)  // M above the diagonal blocks stays zero
        *reinterpret_cast<uint4*>(sm + M1 + 16 * e) = make_uint4(0, 0, 0, 0);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tq = tmem + (static_cast<uint32_t>(quad * 32) << 16);

    // one thread; S comes apart from the rest, as the outputs use its tile
    auto load_keys = [&](const Item& x) {
        mbar_arrive_expect_tx(&bars[0], 32768);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            tma_load_4d(sm + KQ + p * 16384, &tm.k, p * 64, x.hk, x.tt, x.tb, &bars[0]);
            tma_load_4d(sm + KQ + p * 16384 + 8192, &tm.q, p * 64, x.hk, x.tt, x.tb, &bars[0]);
        }
    };
    auto load_head = [&](const Item& x, int h) {
        mbar_arrive_expect_tx(&bars[1], 4 * 16384);
        mbar_arrive_expect_tx(&bars[2], 65536);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            tma_load_4d(sm + VT + p * 8192, &tm.vt, p * 64, h, x.tt, x.tb, &bars[1]);
            tma_load_4d(sm + DL + p * 8192, &tm.dvl, p * 64, h, x.tt, x.tb, &bars[1]);
            tma_load_4d(sm + DV + p * 16384, &tm.dv, p * 64, h, x.tt, x.tb, &bars[1]);
            tma_load_4d(sm + DV + p * 16384 + 8192, &tm.d_o, p * 64, h, x.tt, x.tb, &bars[1]);
            tma_load_3d(sm + GB + p * 16384, &tm.g, p * 64, 0, (int)(x.n * a.H + h), &bars[2]);
        }
    };
    auto load_s = [&](const Item& x, int h) {
#pragma unroll
        for (int p = 0; p < 2; ++p)
            tma_load_3d(sm + SB + p * 16384, &tm.s, p * 64, 0, (int)(x.n * a.H + h), &bars[2]);
    };
    Item cur = item(blockIdx.x);
    if (tid == 0 && cur.cr.valid > 0) {
        load_keys(cur);
        load_head(cur, cur.hk * rep);
        load_s(cur, cur.hk * rep);
    }
    int keys_in = 1, heads_in = 1;  // loads issued (thread 0), to drain after an abort
    const GateVec gv{sm + VEC, 16};
    float* bt = reinterpret_cast<float*>(sm + BT);
    float* rec = reinterpret_cast<float*>(sm + REC);
    float* cs = reinterpret_cast<float*>(sm + CS);
    float* rows = cs;
    float* gs = reinterpret_cast<float*>(sm + GS);
    // gate vectors, record and the chains' sums of a head: warps 8 .. 14, under the loads
    auto head_scalars = [&](const Item& x, int h) {
        const ChunkRows& cr = x.cr;
        const long long n = x.n;
        if (warp == 8) {
            float ga[2], gb[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e;
                const bool in = t < cr.valid;
                ga[e] = in ? a.alpha_log[(cr.row0 + t) * a.H + h] : 0.f;
                gb[e] = in ? a.beta[(cr.row0 + t) * a.H + h] : 0.f;
            }
            scan_gates<false>(gv, bt, nullptr, a.scale, ga, gb, lane);
        } else if (warp == 9) {
            const float4* src = reinterpret_cast<const float4*>(a.blk + ((size_t)n * a.H + h) * kBwdBytes + kBwdImg);
            float4 v[(kBwdRecBytes / 16 + 31) / 32];
#pragma unroll
            for (int e = 0; e < (int)(kBwdRecBytes / 16 + 31) / 32; ++e)
                if (lane + 32 * e < (int)kBwdRecBytes / 16) v[e] = src[lane + 32 * e];
#pragma unroll
            for (int e = 0; e < (int)(kBwdRecBytes / 16 + 31) / 32; ++e)
                if (lane + 32 * e < (int)kBwdRecBytes / 16) reinterpret_cast<float4*>(rec)[lane + 32 * e] = v[e];
        } else if (warp >= 10 && warp < 14) {
            const float* from = warp == 10 ? a.po : warp == 11 ? a.px : warp == 12 ? a.pb : a.pw;
            const float2* p = reinterpret_cast<const float2*>(from + ((size_t)n * a.H + h) * SL * 4 * kChunk) + lane;
            float2 t = make_float2(0.f, 0.f);
            for (int k = 0; k < 4 * SL; k += 8) {  // SL is 2 or 4
                float2 v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = p[(k + e) * 32];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    t.x += v[e].x;
                    t.y += v[e].y;
                }
            }
            reinterpret_cast<float2*>(gs + 64 * (warp - 10))[lane] = t;
        } else if (warp == 14) {
            float end = a.gs[((size_t)n * a.H + h) * SL * 16 + lane];
            if (SL == 4) end += a.gs[((size_t)n * a.H + h) * SL * 16 + 32 + lane];
#pragma unroll
            for (int o = 16; o; o >>= 1) end += __shfl_xor_sync(0xffffffffu, end, o);
            if (lane == 0) gs[256] = end;
        }
    };
    if (cur.cr.valid > 0) head_scalars(cur, cur.hk * rep);
    bool ok = true;
    int u = 0;  // heads processed: the phase of their barriers
    for (int it = 0; cur.cr.valid > 0; ++it) {
        const ChunkRows cr = cur.cr;
        const int hk = cur.hk;
        const Item nx = item(blockIdx.x + (long long)(it + 1) * gridDim.x);
        if (a.cu_s && cr.valid < kChunk) {
            ok = wait_bar(&bars[0], it & 1, abort_flag);
            // K and Q rows behind the sequence meet zeros of M: make them zero
            for (int e = tid; e < 128 * 16; e += kThreads) {
                const int r = e >> 4, p = e & 15;
                if ((r & 63) >= cr.valid)
                    *reinterpret_cast<uint4*>(sm + KQ + (p >> 3) * 16384 + sw128_off(r, p & 7)) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncthreads();
        }
        if (warp == 0) {  // [K; Q] K^T
            ok = wait_bar(&bars[0], it & 1, abort_flag) && ok;
            tc_fence_after_sync();
            __syncwarp();
            constexpr uint32_t id = idesc_bf16(128, 64, false, false);
            const uint64_t d0 = smem_desc(sbase + KQ, 16, 1024, kSw128);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const uint64_t d = d0 + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4);
                mma_bf16_elect(tmem + TM_G, d, d, id, ks > 0);
            }
        }
        for (int hh = 0; hh < rep; ++hh, ++u) {
            const int h = hk * rep + hh;
            if (warp == 0) {
                ok = wait_bar(&bars[1], u & 1, abort_flag) && ok;
                tc_fence_after_sync();
                __syncwarp();
                constexpr uint32_t id = idesc_bf16(128, 64, false, false);
                const uint64_t da = smem_desc(sbase + DV, 16, 1024, kSw128);
                const uint64_t db = smem_desc(sbase + VT, 16, 1024, kSw128);
                const uint64_t dl = smem_desc(sbase + DL, 16, 1024, kSw128);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t ka = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
                    const uint32_t kb = ((ks >> 2) * 8192 + (ks & 3) * 32) >> 4;
                    mma_bf16_elect(tmem + TM_P, da + ka, db + kb, id, ks > 0);
                    // lanes 0..63 only: rows 64.. of this operand are whatever lies behind it
                    mma_bf16_elect(tmem + TM_PL, dl + kb, db + kb, id, ks > 0);
                }
                mma_commit_elect(&bars[3]);
            }
            ok = wait_bar(&bars[3], u & 1, abort_flag) && ok;
            if (!(ok = __syncthreads_and(ok))) break;
            tc_fence_after_sync();
            // ---- rows of -M2 (lanes 0..63) and M1, and the sums of Z: a warp takes 32 rows and one
            // of the column blocks on or left of their diagonal blocks (two, or four)
            {
                const int r = (quad & 1) * 32 + lane, R = r >> 4, I = warp >> 2;
                const bool m1 = quad >= 2, live = r < cr.valid, diag = I >= 2 * (quad & 1);
                if ((quad & 1) || I < 2) {
                    const float lead = m1 ? a.scale : 1.f;
                    const float ph = gv.at(kP, r), pl = gv.at(kPlo, r), ep = expf(ph);
                    float off = lead * fmaf(ep, pl, ep);
                    // whole blocks between this column block and the row's
                    if (R > I + 1) off *= bt[I + 1];
                    if (R > I + 2) off *= bt[I + 2];
                    const int last = I == R ? (r & 15) : I < R ? 16 : -1;  // columns before this one count
                    float g[16], p[16], q[16];
                    tmem_ld16(tq + TM_G + 16 * I, g);
                    tmem_ld16(tq + TM_P + 16 * I, p);
                    if (!m1) tmem_ld16(tq + TM_PL + 16 * I, q);
                    tmem_wait_ld();
                    float sum = 0.f;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const float4 s4 = gv.get4(kSbeta, 4 * I + y);
                        float f[4] = {off * s4.x, off * s4.y, off * s4.z, off * s4.w};
                        if (diag) {  // the warp's rows include this block's diagonal (__expf: 1e-6 at e^-16)
                            const float4 p4 = gv.get4(kP, 4 * I + y), l4 = gv.get4(kPlo, 4 * I + y);
                            const float4 b4 = gv.get4(kBeta, 4 * I + y);
                            const float pv[4] = {p4.x, p4.y, p4.z, p4.w}, lv[4] = {l4.x, l4.y, l4.z, l4.w};
                            const float bv[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float d = lead * bv[e] * __expf((ph - pv[e]) + (pl - lv[e]));
                                f[e] = I == R ? d : f[e];
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = 4 * y + e;
                            const bool in = live && (m1 && I == R ? j <= last : j < last);
                            const float t = m1 ? p[j] : -(p[j] + q[j]);
                            p[j] = in ? f[e] * t : 0.f;
                            // Z, without the diagonal (M1's own: a token's decay does not act on itself)
                            g[j] = live && j < last ? p[j] * g[j] : 0.f;
                            sum += g[j];
                        }
                    }
                    uint8_t* dst = sm + (m1 ? M1 : M2);
                    st_bf16x8(dst + sw128_off(r, 2 * I), p);
                    st_bf16x8(dst + sw128_off(r, 2 * I + 1), p + 8);
                    // sums of 16 columns over 16 rows, column lane % 16 in each lane: halve the
                    // columns a lane holds per step
                    auto over_rows = [&](float (&v)[16]) {
#pragma unroll
                        for (int w = 8; w >= 1; w >>= 1) {
                            const bool up = lane & w;
#pragma unroll
                            for (int j = 0; j < w; ++j) {
                                const float other = __shfl_xor_sync(0xffffffffu, up ? v[j] : v[j + w], w);
                                v[j] = (up ? v[j + w] : v[j]) + other;
                            }
                        }
                        return v[0];
                    };
                    if (diag) {  // of column i, what the rows from i on hold before it
                        float before = 0.f;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            p[j] = I == R && j <= (r & 15) ? before : 0.f;
                            before += g[j];
                        }
                        const float x = over_rows(p);
                        if (I == R) cs[kCsDiag + (m1 ? 64 : 0) + r] = x;
                    }
                    cs[kCsCols + 128 * quad + (lane >> 4) * 64 + 16 * I + (lane & 15)] = over_rows(g);
                    rows[I * 128 + quad * 32 + lane] = sum;
                }
                tc_fence_before_sync();
            }
            // ---- Diag(D) dv (negated), Diag(Dq) dO, Diag(gam) Vtilde in place
#pragma unroll
            for (int e = tid; e < 3 * 64 * 16; e += kThreads) {
                const int which = e >> 10, r = (e >> 4) & 63, c = e & 15;
                uint8_t* at = which == 0   ? sm + DV + (c >> 3) * 16384 + sw128_off(r, c & 7)
                              : which == 1 ? sm + DV + 8192 + (c >> 3) * 16384 + sw128_off(r, c & 7)
                                           : sm + VT + (c >> 3) * 8192 + sw128_off(r, c & 7);
                const float f = which == 0 ? -rec[kRecD + r] : which == 1 ? rec[kRecDq + r] : rec[kRecGam + r];
                float x[8];
                unpack_bf16x8(*reinterpret_cast<const uint4*>(at), x);
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] *= f;
                st_bf16x8(at, x);
            }
            fence_proxy_async_smem();
            __syncthreads();
            tc_fence_after_sync();
            if (warp == 0) {
                ok = wait_bar(&bars[2], u & 1, abort_flag);
                __syncwarp();
                constexpr uint32_t ids = idesc_bf16(64, 128, false, false);   // rows . state^T
                constexpr uint32_t idm = idesc_bf16(64, 128, false, true);    // M . rows
                constexpr uint32_t idt = idesc_bf16(64, 128, true, true);     // M^T . rows
                const uint64_t dv = smem_desc(sbase + DV, 16, 1024, kSw128), dO_ = dv + (8192 >> 4);
                const uint64_t vt = smem_desc(sbase + VT, 16, 1024, kSw128);
                const uint64_t ds = smem_desc(sbase + SB, 16, 1024, kSw128);
                const uint64_t dg = smem_desc(sbase + GB, 16, 1024, kSw128);
                const uint64_t km = smem_desc(sbase + KQ, 16384, 1024, kSw128);         // K, Q as B, MN-major
                const uint64_t qm = smem_desc(sbase + KQ + 8192, 16384, 1024, kSw128);
                const uint64_t m1 = smem_desc(sbase + M1, 16, 1024, kSw128), m1t = smem_desc(sbase + M1, 8192, 1024, kSw128);
                const uint64_t m2 = smem_desc(sbase + M2, 16, 1024, kSw128), m2t = smem_desc(sbase + M2, 8192, 1024, kSw128);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint32_t ka = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
                    const uint32_t kb = ((ks >> 2) * 8192 + (ks & 3) * 32) >> 4;
                    mma_bf16_elect(tmem + TM_Q, dO_ + ka, ds + ka, ids, hh > 0 || ks > 0);
                    mma_bf16_elect(tmem + TM_K, dv + ka, ds + ka, ids, hh > 0 || ks > 0);
                    mma_bf16_elect(tmem + TM_K, vt + kb, dg + ka, ids, 1);
                }
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    mma_bf16_elect(tmem + TM_Q, m1 + ks * 2, km + ks * 128, idm, 1);
                    mma_bf16_elect(tmem + TM_K, m2 + ks * 2, km + ks * 128, idm, 1);
                    mma_bf16_elect(tmem + TM_K, m2t + ks * 128, km + ks * 128, idt, 1);
                    mma_bf16_elect(tmem + TM_K, m1t + ks * 128, qm + ks * 128, idt, 1);
                }
                mma_commit_elect(&bars[4]);
            } else if (warp == 1) {
                // ---- the head's gate gradients: every sum over the terms that count, none taken off
                float c[2], b[2], w_[2], x[3][2], col[2] = {0.f, 0.f};
                const float end = gs[256];
                const int blk = lane >> 3;  // of this lane's two tokens
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 2 * lane + e;
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        x[k][e] = k < blk ? rows[k * 128 + r] + rows[k * 128 + 64 + r] : 0.f;
                        const int R = k + 1;
                        const float* y = cs + kCsCols + (R >> 1) * 128 + (R & 1) * 64 + r;
                        if (R > blk) col[e] += y[0] + y[256];
                    }
                    c[e] = gs[r] - gs[64 + r];
                    b[e] = gs[128 + r];
                    w_[e] = gs[192 + r];
                    if (r >= cr.valid) c[e] = w_[e] = 0.f;
                }
                float pre = w_[0] + w_[1];  // sums over the lanes up to this one
                float s = c[0] + c[1];      // ... from this one on
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float y = __shfl_up_sync(0xffffffffu, pre, o);
                    const float z = __shfl_down_sync(0xffffffffu, s, o);
                    if (lane >= o) pre += y;
                    if (lane + o < 32) s += z;
                }
                pre = __shfl_up_sync(0xffffffffu, pre, 1);  // of the lanes before, of the lanes behind
                s = __shfl_down_sync(0xffffffffu, s, 1);
                if (lane == 0) pre = 0.f;
                if (lane == 31) s = 0.f;
                // the same inside the block: columns before the token, rows from it on
                float cpre = col[0] + col[1], row[2], rsuf;
#pragma unroll
                for (int e = 0; e < 2; ++e) row[e] = x[0][e] + x[1][e] + x[2][e];
                rsuf = row[0] + row[1];
                float b0 = x[0][0] + x[0][1], b1 = x[1][0] + x[1][1];  // whole blocks, of columns 0 .. 15, 16 .. 31
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) {
                    const float y = __shfl_up_sync(0xffffffffu, cpre, o, 8);
                    const float z = __shfl_down_sync(0xffffffffu, rsuf, o, 8);
                    if ((lane & 7) >= o) cpre += y;
                    if ((lane & 7) + o < 8) rsuf += z;
                    b0 += __shfl_xor_sync(0xffffffffu, b0, o);
                    b1 += __shfl_xor_sync(0xffffffffu, b1, o);
                }
                cpre = __shfl_up_sync(0xffffffffu, cpre, 1, 8);
                rsuf = __shfl_down_sync(0xffffffffu, rsuf, 1, 8);
                if ((lane & 7) == 0) cpre = 0.f;
                if ((lane & 7) == 7) rsuf = 0.f;
                const float b20 = __shfl_sync(0xffffffffu, b0, 16), b30 = __shfl_sync(0xffffffffu, b0, 24);
                const float b31 = __shfl_sync(0xffffffffu, b1, 24);
                const float whole = blk == 1 ? b20 + b30 : blk == 2 ? b30 + b31 : 0.f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 2 * lane + e;
                    if (r < cr.valid) {
                        const size_t at = (size_t)(cr.row0 + r) * a.H + h;
                        const float pairs = cs[kCsDiag + r] + cs[kCsDiag + 64 + r] + whole +
                                            (e == 0 ? cpre : cpre + col[0]) +
                                            (e == 0 ? row[0] + (row[1] + rsuf) : row[1] + rsuf);
                        float y = (e == 0 ? c[0] + (c[1] + s) : c[1] + s) + (e == 0 ? pre : pre + w_[0]) + end +
                                  pairs;
                        // nothing enters a sequence's first token from no state: its decay has no effect
                        if (r == 0 && cr.first && !a.S0) y = 0.f;
                        a.dalpha_log[at] = y;
                        a.dbeta[at] = b[e];
                    }
                }
            }
            ok = wait_bar(&bars[4], u & 1, abort_flag) && ok;
            if (!(ok = __syncthreads_and(ok))) break;
            tc_fence_after_sync();
            if (hh + 1 < rep) {
                if (tid == 0) {
                    load_head(cur, h + 1);
                    load_s(cur, h + 1);
                    ++heads_in;
                }
                head_scalars(cur, h + 1);
            }
        }
        if (!ok) break;
        // the next chunk's tiles are on their way while this one's dq and dk leave
        if (tid == 0 && nx.cr.valid > 0) {
            load_keys(nx);
            load_head(nx, nx.hk * rep);
            ++keys_in;
            ++heads_in;
        }
        // ---- dq, dk: bf16 through the tile of S; a warp 64 columns of 16 rows of one of them
        const int r0 = quad * 16 + (lane >> 2), pc = (lane & 3) * 4, half = (warp >> 2) & 1, w = warp >> 3;
        float x[32];
        tmem_ld_16x256<8>(tq + (w ? TM_K : TM_Q) + 64 * half, x);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<uint32_t*>(sm + SB + w * 16384 + half * 8192 + sw128_off(r0 + 8 * e, c) + pc) =
                    pack_bf16(x[4 * c + 2 * e], x[4 * c + 2 * e + 1]);
        fence_proxy_async_smem();
        tc_fence_before_sync();
        __syncthreads();
        if (!a.cu_s || cr.valid == kChunk) {
            if (tid == kThreads - 32) {  // a warp with nothing else to do until the next rows
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    tma_store_4d(&tm.dq, p * 64, hk, cur.tt, cur.tb, sm + SB + p * 8192);
                    tma_store_4d(&tm.dk, p * 64, hk, cur.tt, cur.tb, sm + SB + 16384 + p * 8192);
                }
                bulk_commit_group();
                bulk_wait_group_read<0>();
            }
        } else {
            for (int e = tid; e < 2 * 64 * 16; e += kThreads) {
                const int w = e >> 10, r = (e >> 4) & 63, c = e & 15;
                if (r < cr.valid)
                    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(w ? a.dk : a.dq) +
                                              ((size_t)(cr.row0 + r) * a.Hk + hk) * D + 8 * c) =
                        *reinterpret_cast<const uint4*>(sm + SB + w * 16384 + (c >> 3) * 8192 + sw128_off(r, c & 7));
            }
        }
        if (nx.cr.valid > 0) {
            if (a.cu_s && cr.valid < kChunk) __syncthreads();  // the tile has been read
            if (tid == kThreads - 32) {
                fence_proxy_async_smem();
                load_s(nx, nx.hk * rep);
            }
            head_scalars(nx, nx.hk * rep);
        }
        cur = nx;
    }
    if (!ok && tid == 0) {
        // after an abort: copies in flight land before shared memory is released
        (void)mbar_wait(&bars[0], (keys_in - 1) & 1);
        (void)mbar_wait(&bars[1], (heads_in - 1) & 1);
        (void)mbar_wait(&bars[2], (heads_in - 1) & 1);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (tid == 0 && *abort_flag) atomicOr(a.status + 1, 1u);
    if (warp == 0) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

cudaError_t launch_rebuild_tc(const Args& a, int ns, cudaStream_t s);
cudaError_t launch_reverse_tc(const Args& a, int ns, cudaStream_t s);

cudaError_t launch_bwd_tc(const Args& a, cudaStream_t s)
{
    cudaError_t e;
    if ((e = launch_operands_tc(a, s, true, 0, 0)) != cudaSuccess) return e;
    if ((e = launch_rebuild_tc(a, a.ns, s)) != cudaSuccess) return e;
    if ((e = launch_reverse_tc(a, a.ns, s)) != cudaSuccess) return e;
    const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
    GradMaps m;
    if (!make_rows_map(&m.q, a.q, a, a.Hk, 64, sw) || !make_rows_map(&m.k, a.k, a, a.Hk, 64, sw) ||
        !make_rows_map(&m.vt, a.vt, a, a.H, 64, sw) || !make_rows_map(&m.d_o, a.d_o, a, a.H, 64, sw) ||
        !make_rows_map(&m.dv, a.dv, a, a.H, 64, sw) || !make_rows_map(&m.dvl, a.dvl, a, a.H, 64, sw) ||
        !make_rows_map(&m.dq, a.dq, a, a.Hk, 64, sw) || !make_rows_map(&m.dk, a.dk, a, a.Hk, 64, sw) ||
        !make_states_map(&m.s, a.sb, a, 64, sw) || !make_states_map(&m.g, a.gb, a, 64, sw))
        return cudaErrorInvalidValue;
    if ((e = cudaFuncSetAttribute(grads_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)BYTES)) !=
        cudaSuccess)
        return e;
    const long long blocks = chunks(a) * a.Hk;
    if (blocks == 0) return cudaSuccess;
    ProfScope ps(kGdrBwdGrads, s);
    int dev = 0, sms = 148;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    grads_kernel<<<(unsigned)(blocks < sms ? blocks : sms), kThreads, BYTES, s>>>(m, a, blocks);
    return cudaGetLastError();
}

}  // namespace gdr
}  // namespace mdn
