// The chunk operands of the gated delta rule on sm_100a (formulas and layout in
// gdr_tc.cuh): one CTA of 128 threads per chunk and head at a time, three CTAs
// per SM, so that one CTA's dependent phases run under the others'.
//
//   1  [K; Q] by TMA; G = [K; Q] K^T on tcgen05 (M 128, N 64, K = d): exact
//      products of the inputs, fp32 sums; the next chunk's load follows at once
//   2  TMEM lane r is row r of A (lanes 0..63) or of Att (lanes 64..127).  Warp w < 2
//      writes rows 32 w .. of A to shared memory in fp32 and, alone, inverts
//      its two 16 x 16 diagonal blocks (a lane per column, forward substitution
//      in fp32 with x in registers) and joins them, T_10 = -T_11 A_10 T_00; warps 2 and 3
//      write Att to the block image and scan the next chunk's gates meanwhile
//   3  the join of the two 32 x 32 halves, by all four warps
//   4  T rounded to two bf16 terms into the image; one bulk store
//
// Bound by the latency of these phases: 11k cycles per chunk with three CTAs per SM,
// which is what shared memory admits; 8 x 4096 tokens of 16 heads take 107 us, of which
// their 482 MB of inputs and blocks need 75 at the copy rate.
//
// The decays L need care: differences of long sums of alpha_log lose the
// digits that exp then needs.  Inside a 16 x 16 diagonal block they are
// differences of sums of at most 16 terms held as two floats; off the diagonal
// they are products of factors that are each an exponential of one such sum
// (exp(p_r) to the left edge of row block R, the whole blocks between, exp(s_i)
// to the right edge of column block I), so no exponential per element either.
// (fp64 for the sums measured 3.6k cycles for the scan and 7k for the rows.)
// alpha_log below -1e4 (alpha = 0 in fp32 already at -104) counts as -1e4, so
// that -inf resets the state instead of giving inf - inf.
#include "gdr_tc.cuh"

namespace mdn {
namespace gdr {
namespace {

using namespace sm100;
using namespace tc;
using inter::wait_bar;

constexpr int kThreads = 128;
constexpr int LDA = 68;  // leading dimension of the fp32 matrix (16-byte rows, no bank conflicts)

template <int D, bool BWD>
struct Lay {
    static constexpr uint32_t IMG_BYTES = BWD ? kBwdImg : kBlkImg;
    static constexpr int CTAS = BWD ? 2 : 3;  // per SM
    static constexpr uint32_t KQ = 0;                        // D/64 panels of [K; Q], 128 rows x 128 B
    static constexpr uint32_t IMG = KQ + (D / 64) * 16384;   // the images being built
    static constexpr uint32_t AM = IMG + IMG_BYTES;          // A, then T; gate vectors of odd chunks in
                                                             // the rows' padding
    static constexpr uint32_t VEC = AM + 64 * LDA * 4;       // gate vectors of even chunks
    static constexpr uint32_t BTOT = VEC + 4 * 256;          // [2][4] exp of a block's sum
    static constexpr uint32_t BARS = BTOT + 32;
    static constexpr uint32_t MISC = BARS + 16;
    static constexpr uint32_t BYTES = MISC + 32;
    static_assert(BARS % 8 == 0 && AM % 16 == 0, "alignment");
    static_assert(CTAS * (BYTES + 1024) <= 233472, "CTAs per SM");
};

struct OpArgs {
    Args a;
    uint8_t* blk;
    const int* chunk_order;
    unsigned* ready;
    int total;  // chunk-heads
    int reserve, limit;
};

// A chunk-head of the work order: the first chunks of every chain come first.
struct Item {
    int n, h, valid, b, t;  // chunk of the call, head, tokens; batch row and token of the TMA maps
    long long row0;
};
__device__ __forceinline__ Item item(const OpArgs& o, int i)
{
    const Args& a = o.a;
    Item x;
    const int r = i / a.H;
    x.h = i - r * a.H;
    if (a.cu_s) {
        x.n = o.chunk_order[r];
        const ChunkRows cr = chunk_rows(a, x.n);
        x.row0 = cr.row0;
        x.valid = cr.valid;
        x.b = 0;
        x.t = (int)cr.row0;
    } else {
        const int c = r / a.B;
        x.b = r - c * a.B;
        x.n = x.b * a.NT + c;
        x.t = c * kChunk;
        x.row0 = (long long)x.b * a.T + x.t;
        x.valid = min(kChunk, a.T - x.t);
    }
    return x;
}

// 16 x 16 products of fp32 matrices in shared memory (leading dimension LDA), one warp:
// the 16-row blocks are below tcgen05's smallest M, so they take the warp-level bf16
// instruction, each factor as two bf16 terms and three of the four term products
// (2^-16 relative, below the rounding of T to two terms).  In FP32 multiply-adds these
// joins were half of the kernel's instructions.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// acc[n] (columns 8 n ..) += X (16 x 16 at x) Y (16 x 16 at y)
__device__ __forceinline__ void block_mm(float (&acc)[2][4], const float* x, const float* y, int lane)
{
    const int g = lane >> 2, t = lane & 3;
    uint32_t ah[4], al[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = *reinterpret_cast<const float2*>(x + (g + 8 * (i & 1)) * LDA + 2 * t + 8 * (i >> 1));
        split2(v.x, v.y, ah[i], al[i]);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        uint32_t bh[2], bl[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float* p = y + (2 * t + 8 * i) * LDA + 8 * n + g;
            split2(p[0], p[LDA], bh[i], bl[i]);
        }
        mma_16816(acc[n], ah, bh[0], bh[1]);
        mma_16816(acc[n], ah, bl[0], bl[1]);
        mma_16816(acc[n], al, bh[0], bh[1]);
    }
}
// dst (16 x 16) = f acc
__device__ __forceinline__ void block_st(float* dst, const float (&acc)[2][4], float f, int lane)
{
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float2*>(dst + (g + 8 * h) * LDA + 8 * n + 2 * t) =
                make_float2(f * acc[n][2 * h], f * acc[n][2 * h + 1]);
}
__device__ __forceinline__ void block_zero(float (&acc)[2][4])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j >> 2][j & 3] = 0.f;
}

template <int D, bool BWD>
__global__ void __launch_bounds__(kThreads, BWD ? 2 : 3)
operands_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const OpArgs o)
{
    using L = Lay<D, BWD>;
    constexpr uint32_t kBlock = BWD ? kBwdBytes : kBlkBytes;
    const Args& a = o.a;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_launch_dependents();
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BARS);  // [0] load, [1] product
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC + 4);
    float* Am = reinterpret_cast<float*>(sm + L::AM);
    int* slot = reinterpret_cast<int*>(sm + L::MISC + 8);  // [4] work items of iterations k, k + 1, ...
    auto vec = [&](int k) { return k & 1 ? GateVec{sm + L::AM + 256, LDA * 4} : GateVec{sm + L::VEC, 16}; };
    auto btot = [&](int k) { return reinterpret_cast<float*>(sm + L::BTOT) + 4 * (k & 1); };

    if (tid == 0) {
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
        mbar_fence_init();
        *abort_flag = 0;
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, 64);
        tmem_relinquish();
    }
    // the blocks above the diagonal of every image stay zero
    for (int e = tid; e < (int)L::IMG_BYTES / 16; e += kThreads)
        *reinterpret_cast<uint4*>(sm + L::IMG + 16 * e) = make_uint4(0, 0, 0, 0);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    auto load = [&](const Item& x) {  // one thread
        const int hk = x.h / (a.H / a.Hk);
        mbar_arrive_expect_tx(&bars[0], (D / 64) * 16384);
#pragma unroll
        for (int p = 0; p < D / 64; ++p) {
            tma_load_4d(sm + L::KQ + p * 16384, &tm_k, p * 64, hk, x.t, x.b, &bars[0]);
            tma_load_4d(sm + L::KQ + p * 16384 + 8192, &tm_q, p * 64, hk, x.t, x.b, &bars[0]);
        }
    };
    float ga[2] = {0.f, 0.f}, gb[2] = {0.f, 0.f};  // warp 2: gates of the next chunk to scan
    auto load_gates = [&](const Item& x) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            const bool in = t < x.valid;
            ga[e] = in ? a.alpha_log[(x.row0 + t) * a.H + x.h] : 0.f;
            gb[e] = in ? a.beta[(x.row0 + t) * a.H + x.h] : 0.f;
        }
    };
    auto rec_of = [&](const Item& x) {
        return reinterpret_cast<float*>(o.blk + ((size_t)x.n * a.H + x.h) * kBlock + L::IMG_BYTES);
    };
    // Work items come from a counter, one thread (tid 96) taking each two iterations ahead.
    // Chunks with no tokens (a packed call's bound on its chunks) end the work order.
    int taken = 0, limit = 1 << 30;
    auto take = [&]() -> int {
        // stop at the limit, provided that a CTA without one is at work on the rest
        if (taken >= limit && *reinterpret_cast<volatile unsigned*>(o.ready + o.total + 1)) return o.total;
        ++taken;
        const unsigned c = atomicAdd(o.ready + o.total, 1u);
        return c < (unsigned)o.total ? (int)c : o.total;
    };
    if (tid == 96) {
        uint32_t smid;
        asm volatile("mov.u32 %0, %%smid;" : "=r"(smid));
        if ((int)smid < o.reserve) limit = o.limit;
        else if (o.reserve) atomicAdd(o.ready + o.total + 1, 1u);
        slot[0] = take();
        slot[1] = slot[0] < o.total ? take() : o.total;
    }
    __syncthreads();
    bool more = false, pending = false;
    Item x, nx;
    if (slot[0] < o.total) {
        x = item(o, slot[0]);
        more = x.valid > 0;
    }
    if (more) {
        if (tid == 96) {
            load(x);
            pending = true;
        }
        if (warp == 2) {
            load_gates(x);
            scan_gates<BWD>(vec(0), btot(0), rec_of(x), a.scale, ga, gb, lane);
        }
    }
    bool next = more && slot[1] < o.total;
    if (next) {
        nx = item(o, slot[1]);
        next = nx.valid > 0;
        if (next && warp == 2) load_gates(nx);
    }
    // thread 0: the block of the chunk before has been stored; say so
    unsigned* done = nullptr;
    auto publish = [&]() {
        if (!done) return;
        fence_proxy_async_global();
        st_release_gpu(done, 1u);
        done = nullptr;
    };
    __syncthreads();
    for (int k = 0; more; ++k) {
        const GateVec gv = vec(k);
        const float* bt = btot(k);
        bool ok = true;
        if (a.cu_s && x.valid < kChunk) {
            // rows behind the sequence hold the next one's (or anything): make them zero, so
            // that A and Att are zero there (a batch's rows past T were read as zeros)
            ok = wait_bar(&bars[0], k & 1, abort_flag);
            for (int e = tid; e < 128 * 8 * (D / 64); e += kThreads) {
                const int r = e & 127, c = e >> 7;
                if ((r & 63) >= x.valid)
                    *reinterpret_cast<uint4*>(sm + L::KQ + (c >> 3) * 16384 + sw128_off(r, c & 7)) =
                        make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncthreads();
        }
        if (warp == 0) {
            ok = wait_bar(&bars[0], k & 1, abort_flag) && ok;
            tc_fence_after_sync();
            __syncwarp();
            constexpr uint32_t id = idesc_bf16(128, 64, false, false);
            const uint64_t d0 = smem_desc(sbase + L::KQ, 16, 1024, kSw128);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint64_t d = d0 + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4);
                mma_bf16_elect(tmem, d, d, id, ks > 0);
            }
            mma_commit_elect(&bars[1]);
            if (lane == 0) {  // the last image has left (overlapped: has been written)
                if (done) {
                    bulk_wait_group<0>();
                    publish();
                } else {
                    bulk_wait_group_read<0>();
                }
            }
            __syncwarp();
        }
        ok = wait_bar(&bars[1], k & 1, abort_flag) && ok;
        if (!__syncthreads_and(ok)) break;
        tc_fence_after_sync();
        int c2 = o.total;
        if (tid == 96) {
            pending = next;
            if (next) {
                load(nx);
                c2 = take();  // waited for after the rows below
            }
        }
        // ---- rows of A and Att, the diagonal 32 x 32 halves of T
        {
            const int r = tid & 63, R = r >> 4;
            const bool att = warp >= 2, low = lane < 16;
            const uint32_t t0 = tmem + (static_cast<uint32_t>(warp * 32) << 16);
            const float ph = gv.at(kP, r), pl = gv.at(kPlo, r);
            // forward: column i carries beta_i; backward: row r of A carries beta_r
            const float lead = att ? a.scale : BWD ? gv.at(kBeta, r) : 1.f;
            const float ep = expf(ph);
            float off = lead * fmaf(ep, pl, ep);  // exp(p_r), then times the whole blocks between
            const int last = (r & 15) + (att ? 1 : 0);  // columns of the diagonal block that count
            auto put = [&](int I, const float (&g)[16]) {
                if (att) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint4 hi, lo;
                        if (BWD) {
                            split8(g + 8 * c, hi, lo);
                            *reinterpret_cast<uint4*>(sm + L::IMG + kBwdAttLo + sw128_off(r, 2 * I + c)) = lo;
                        } else {
                            hi = bf16x8(g + 8 * c);
                        }
                        *reinterpret_cast<uint4*>(sm + L::IMG + kBlkAtt + sw128_off(r, 2 * I + c)) = hi;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4*>(Am + r * LDA + 16 * I + j) =
                            make_float4(g[j], g[j + 1], g[j + 2], g[j + 3]);
                }
            };
            // the two column blocks that hold the diagonal: a lane's own (its factors are the
            // exponentials) and, for lanes 16..31, the one left of it
            const int I0 = (warp & 1) * 2;
            // (__expf: 2 ulp and half an ulp of the argument, 1e-6 at e^-16, below the two-term rounding)
            float fd[16];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 p4 = gv.get4(kP, 4 * R + q), l4 = gv.get4(kPlo, 4 * R + q);
                const float4 b4 = gv.get4(kBeta, 4 * R + q);
                const float pv[4] = {p4.x, p4.y, p4.z, p4.w}, lv[4] = {l4.x, l4.y, l4.z, l4.w};
                const float bv[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    fd[4 * q + e] = (BWD ? lead : lead * bv[e]) * __expf((ph - pv[e]) + (pl - lv[e]));
            }
#pragma unroll
            for (int x2 = 1; x2 >= 0; --x2) {
                const int I = I0 + x2;
                float g[16];
                tmem_ld16(t0 + 16 * I, g);
                tmem_wait_ld();
                const bool own = x2 == 0 ? low : !low;
                const int upto = own ? last : x2 == 0 ? 16 : 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 s4 = gv.get4(kSbeta, 4 * I + q);
                    const float sv[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = 4 * q + e;
                        const float f = own ? fd[j] : off * sv[e];
                        g[j] = j < upto ? g[j] * f : 0.f;  // a select: what is masked may be NaN
                    }
                }
                put(I, g);
                if (x2 == 0 && !low) off *= bt[I];
            }
            // the blocks left of them: no mask, factors exp(p_r) . whole blocks . exp(s_i)
            if (warp & 1)
#pragma unroll
                for (int I = 1; I >= 0; --I) {
                    float g[16];
                    tmem_ld16(t0 + 16 * I, g);
                    tmem_wait_ld();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 s4 = gv.get4(kSbeta, 4 * I + q);
                        g[4 * q] *= off * s4.x;
                        g[4 * q + 1] *= off * s4.y;
                        g[4 * q + 2] *= off * s4.z;
                        g[4 * q + 3] *= off * s4.w;
                    }
                    put(I, g);
                    off *= bt[I];
                }
        }
        tc_fence_before_sync();
        if (warp < 2) {
            __syncwarp();
            // column c of diagonal block b
            const int b = warp * 2 + (lane >> 4), c = lane & 15;
            float* blk = Am + (16 * b) * LDA + 16 * b;
            float y[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float v = r == c ? 1.f : 0.f;
#pragma unroll
                for (int k4 = 0; k4 < r; k4 += 4) {
                    const float4 w = lds4(blk + r * LDA + k4);
                    const float wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (k4 + e < r) v = fmaf(-wv[e], y[k4 + e], v);
                }
                y[r] = v;
            }
            __syncwarp();
#pragma unroll
            for (int r = 0; r < 16; ++r) blk[r * LDA + c] = y[r];
            __syncwarp();
            // T_10 = -T_11 (A_10 T_00); the product in brackets above the diagonal
            float* lo = Am + (32 * warp) * LDA + 32 * warp;
            float acc[2][4];
            block_zero(acc);
            block_mm(acc, lo + 16 * LDA, lo, lane);
            block_st(lo + 16, acc, 1.f, lane);
            __syncwarp();
            block_zero(acc);
            block_mm(acc, lo + 16 * LDA + 16, lo + 16, lane);
            block_st(lo + 16 * LDA, acc, -1.f, lane);
        } else if (warp == 2 && next) {
            scan_gates<BWD>(vec(k + 1), btot(k + 1), rec_of(nx), a.scale, ga, gb, lane);
        }
        if (tid == 96) slot[(k + 2) & 3] = c2;
        __syncthreads();
        Item nx2 = nx;
        bool n2 = next && slot[(k + 2) & 3] < o.total;
        if (n2) {
            nx2 = item(o, slot[(k + 2) & 3]);
            n2 = nx2.valid > 0;
            if (n2 && warp == 2) load_gates(nx2);
        }
        // ---- the two halves joined: M = A_10 T_00 (above the diagonal), T_10 = -T_11 M.
        // A warp takes 16 x 16 of the result; the 16 x 16 blocks above T_00's and T_11's own
        // diagonals (scratch, mathematically zero) are skipped.
        {
            const int u = warp >> 1, v = warp & 1;
            float acc[2][4];
            block_zero(acc);  // rows 16 v .., columns 16 u ..
            for (int k = u; k < 2; ++k)
                block_mm(acc, Am + (32 + 16 * v) * LDA + 16 * k, Am + 16 * k * LDA + 16 * u, lane);
            block_st(Am + 16 * v * LDA + 32 + 16 * u, acc, 1.f, lane);
            __syncthreads();
            block_zero(acc);  // rows 16 u .., columns 16 v ..
            for (int k = 0; k <= u; ++k)
                block_mm(acc, Am + (32 + 16 * u) * LDA + 32 + 16 * k, Am + 16 * k * LDA + 32 + 16 * v, lane);
            block_st(Am + (32 + 16 * u) * LDA + 16 * v, acc, -1.f, lane);
        }
        __syncthreads();
        // ---- T in two bf16 terms: 320 pieces of 8 columns on and below the diagonal blocks
#pragma unroll
        for (int it = 0; it < 3; ++it) {
            const int e = tid + kThreads * it;
            if (e < 320) {
                const int R = e < 32 ? 0 : e < 96 ? 1 : e < 192 ? 2 : 3;
                const int l = e - 16 * R * (R + 1), w = 2 * (R + 1), r = 16 * R + l / w, c8 = l % w;
                float z[8];
                const float4 p = lds4(Am + r * LDA + 8 * c8), q = lds4(Am + r * LDA + 8 * c8 + 4);
                z[0] = p.x; z[1] = p.y; z[2] = p.z; z[3] = p.w;
                z[4] = q.x; z[5] = q.y; z[6] = q.z; z[7] = q.w;
                uint4 hi, lo;
                split8(z, hi, lo);
                *reinterpret_cast<uint4*>(sm + L::IMG + kBlkThi + sw128_off(r, c8)) = hi;
                *reinterpret_cast<uint4*>(sm + L::IMG + kBlkTlo + sw128_off(r, c8)) = lo;
            }
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            bulk_store(o.blk + ((size_t)x.n * a.H + x.h) * kBlock, sm + L::IMG, L::IMG_BYTES);
            bulk_commit_group();
            if (o.reserve) done = o.ready + (size_t)x.n * a.H + x.h;
        }
        more = next;
        x = nx;
        next = n2;
        nx = nx2;
    }
    if (tid == 96 && pending) {
        // after an abort: the load in flight must land before shared memory is released
        (void)mbar_wait(&bars[0], 0);
        (void)mbar_wait(&bars[0], 1);
    }
    if (tid == 0) {
        bulk_wait_group_all();
        publish();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (tid == 0 && *abort_flag) atomicOr(a.status + 1, 1u);
    if (warp == 0) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 64);
    }
}

template <int D, bool BWD>
cudaError_t launch_typed(const Args& a, cudaStream_t s, int reserve, int limit)
{
    using L = Lay<D, BWD>;
    CUtensorMap mq, mk;
    if (!make_rows_map(&mq, a.q, a, a.Hk, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_rows_map(&mk, a.k, a, a.Hk, 64, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    int dev = 0, sms = 148;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(operands_kernel<D, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)L::BYTES);
    if (e != cudaSuccess) return e;
    OpArgs o;
    o.a = a;
    o.blk = a.blk;
    o.chunk_order = a.chunk_order;
    o.ready = a.ready;
    o.reserve = reserve;
    o.limit = limit;
    o.total = (int)(chunks(a) * a.H);  // < 2^31
    if (o.total == 0) return cudaSuccess;
    const int grid = o.total < L::CTAS * sms ? o.total : L::CTAS * sms;
    ProfScope ps(kGdrOperands, s);
    operands_kernel<D, BWD><<<grid, kThreads, L::BYTES, s>>>(mq, mk, o);
    return cudaGetLastError();
}

}  // namespace

bool make_rows_map(CUtensorMap* map, const void* base, const Args& a, int heads, int box_d,
                   CUtensorMapSwizzle swizzle, int box_rows)
{
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t T = (cuuint64_t)a.T, B = a.cu_s ? 1 : (cuuint64_t)a.B;
    const cuuint64_t row = (cuuint64_t)heads * a.D * 2;
    cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)heads, T, B};
    cuuint64_t strides[3] = {(cuuint64_t)a.D * 2, row, T * row};
    cuuint32_t box[4] = {(cuuint32_t)box_d, 1, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_states_map(CUtensorMap* map, const void* base, const Args& a, int box_d, CUtensorMapSwizzle swizzle)
{
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t d = (cuuint64_t)a.D;
    cuuint64_t dims[3] = {d, d, (cuuint64_t)(chunks(a) * a.H)};
    cuuint64_t strides[2] = {d * 2, d * d * 2};
    cuuint32_t box[3] = {(cuuint32_t)box_d, (cuuint32_t)a.D, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_operands_tc(const Args& a, cudaStream_t s, bool bwd, int reserve, int limit)
{
    if (bwd) return launch_typed<128, true>(a, s, reserve, limit);
    return a.D == 64 ? launch_typed<64, false>(a, s, reserve, limit)
                     : launch_typed<128, false>(a, s, reserve, limit);
}

}  // namespace gdr
}  // namespace mdn
