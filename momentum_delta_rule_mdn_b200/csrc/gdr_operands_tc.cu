// The chunk operands of the gated delta rule on sm_100a (formulas and layout in
// gdr_tc.cuh): one CTA of 128 threads per chunk and head at a time, three CTAs
// per SM, so that one CTA's dependent phases run under the others'.
//
//   1  [K; Q] by TMA; G = [K; Q] K^T on tcgen05 (M 128, N 64, K = d): exact
//      products of the inputs, fp32 sums
//   2  TMEM lane r: row r of A (lanes 0..63, fp32 to shared memory) and of Att
//      (lanes 64..127, bf16 to the block image); the next chunk's load is issued
//      as soon as G is done
//   3  T = (I + A)^{-1} in fp32 by 16 x 16 blocks: diagonal blocks by forward
//      substitution (a thread per column, x in registers), then pairs to 32,
//      then 64, as -T_11 A_10 T_00
//   4  T rounded to two bf16 terms into the image; one bulk store
//
// The decays L need care: differences of long sums of alpha_log lose the
// digits that exp then needs.  Inside a 16 x 16 diagonal block they are fp64
// differences of sums of at most 16 terms; off the diagonal they are products
// of factors that are each an exponential of one such sum (exp(p_r) to the left
// edge of row block R, the whole blocks between, exp(s_i) to the right edge of
// column block I), so no exponential per element either.  alpha_log below -1e4
// (alpha = 0 in fp32 already at -104) counts as -1e4, so that -inf resets the
// state instead of giving inf - inf.
#include "gdr_tc.cuh"

namespace mdn {
namespace gdr {
namespace {

using namespace sm100;
using namespace tc;
using inter::wait_bar;

constexpr int kThreads = 128;
constexpr int LDA = 68;  // leading dimension of the fp32 matrix (16-byte rows, no bank conflicts)

template <int D>
struct Lay {
    static constexpr uint32_t KQ = 0;                        // D/64 panels of [K; Q], 128 rows x 128 B
    static constexpr uint32_t IMG = KQ + (D / 64) * 16384;   // the block being built
    static constexpr uint32_t AM = IMG + kBlkBytes;          // A, then T
    static constexpr uint32_t VEC = IMG + kBlkTlo;           // gate vectors (1,296 B), before T_lo
    static constexpr uint32_t BARS = AM + 64 * LDA * 4;
    static constexpr uint32_t MISC = BARS + 32;
    static constexpr uint32_t BYTES = MISC + 32;
    static_assert(BARS % 8 == 0 && IMG % 1024 == 0 && AM % 16 == 0, "alignment");
    static_assert(3 * (BYTES + 1024) <= 233472, "three CTAs per SM");
};

struct OpArgs {
    Args a;
    uint8_t* blk;
    const int* chunk_order;
    long long total;  // chunk-heads
};

// Chunk-head `i` of the work order: chunk n of the call, head h (the first chunks
// of every chain come first).
__device__ __forceinline__ void item(const OpArgs& o, long long i, long long& n, int& h)
{
    const Args& a = o.a;
    h = (int)(i % a.H);
    const long long r = i / a.H;
    n = a.cu_s ? (long long)o.chunk_order[r] : r % a.B * a.NT + r / a.B;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 3)
operands_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const OpArgs o)
{
    using L = Lay<D>;
    const Args& a = o.a;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BARS);  // [0] load, [1] product
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC + 4);
    float* Am = reinterpret_cast<float*>(sm + L::AM);
    double* psum = reinterpret_cast<double*>(sm + L::VEC);        // sums inside a block of 16
    float* pexp = reinterpret_cast<float*>(sm + L::VEC + 512);    // exp(p_r)
    float* beta = pexp + 64;
    float* sbeta = beta + 64;                                     // beta_i exp(tot - p_i)
    float* btot = sbeta + 64;                                     // [4] exp of a block's sum

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
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    auto load = [&](long long i) {  // thread 0
        long long n;
        int h;
        item(o, i, n, h);
        const ChunkRows cr = chunk_rows(a, n);
        if (cr.valid <= 0) return false;
        const int hk = h / (a.H / a.Hk);
        const int b = a.cu_s ? 0 : (int)(n / a.NT);
        const int t = a.cu_s ? (int)cr.row0 : (int)(n % a.NT) * kChunk;
        mbar_arrive_expect_tx(&bars[0], (D / 64) * 16384);
#pragma unroll
        for (int p = 0; p < D / 64; ++p) {
            tma_load_4d(sm + L::KQ + p * 16384, &tm_k, p * 64, hk, t, b, &bars[0]);
            tma_load_4d(sm + L::KQ + p * 16384 + 8192, &tm_q, p * 64, hk, t, b, &bars[0]);
        }
        return true;
    };
    bool pending = false;  // thread 0: a load is in flight
    long long i = blockIdx.x;
    if (tid == 0 && i < o.total) pending = load(i);
    // the gates of the chunk, two tokens per lane of warp 0
    float ga[2] = {0.f, 0.f}, gb[2] = {0.f, 0.f};
    auto load_gates = [&](long long j) {
        long long n;
        int h;
        item(o, j, n, h);
        const ChunkRows cr = chunk_rows(a, n);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            const bool in = t < cr.valid;
            ga[e] = in ? a.alpha_log[(cr.row0 + t) * a.H + h] : 0.f;
            gb[e] = in ? a.beta[(cr.row0 + t) * a.H + h] : 0.f;
        }
    };
    if (warp == 0 && i < o.total) load_gates(i);
    uint32_t phase = 0;
    for (; i < o.total; i += gridDim.x) {
        long long n;
        int h;
        item(o, i, n, h);
        const ChunkRows cr = chunk_rows(a, n);
        const long long next = i + gridDim.x;
        if (cr.valid <= 0) {  // an unused chunk of a packed call: uniform for the CTA
            if (tid == 0 && next < o.total) pending = load(next);
            if (warp == 0 && next < o.total) load_gates(next);
            continue;
        }
        float* rec = reinterpret_cast<float*>(sm + L::IMG + kBlkRec);
        if (tid == 0) bulk_wait_group_read<0>();  // the image has left
        if (warp == 0) {
            __syncwarp();
            // sums inside blocks of 16 (8 lanes), fp64
            double p0 = fmax((double)ga[0], -1e4), p1 = p0 + fmax((double)ga[1], -1e4);
            if (ga[0] != ga[0]) p0 = p1 = ga[0];
            if (ga[1] != ga[1]) p1 = ga[1];
            double s = p1;
#pragma unroll
            for (int off = 1; off < 8; off <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, s, off, 8);
                if ((lane & 7) >= off) s += y;
            }
            double before = __shfl_up_sync(0xffffffffu, s, 1, 8);
            if ((lane & 7) == 0) before = 0.0;
            const double q0 = before + p0, q1 = before + p1;
            const double tot = __shfl_sync(0xffffffffu, s, 7, 8);
            double bt[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) bt[b] = __shfl_sync(0xffffffffu, tot, 8 * b);
            const int B = lane >> 3;
            double pre = 0.0, post = 0.0;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (b < B) pre += bt[b];
                if (b > B) post += bt[b];
            }
            const float fpre = expf((float)pre), fpost = expf((float)post);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 2 * lane + e;
                const double q = e ? q1 : q0;
                const float ep = expf((float)q), es = expf((float)(tot - q));
                psum[r] = q;
                pexp[r] = ep;
                beta[r] = gb[e];
                sbeta[r] = gb[e] * es;
            }
            if ((lane & 7) == 0) btot[B] = expf((float)tot);
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 2 * lane + e;
                const float D_ = pexp[r] * fpre;
                rec[kRecD + r] = D_;
                rec[kRecDq + r] = a.scale * D_;
                rec[kRecGam + r] = sbeta[r] * fpost;
            }
            if (lane == 0) rec[kRecB] = expf((float)(bt[0] + bt[1] + bt[2] + bt[3]));
            if (next < o.total) load_gates(next);
        }
        bool ok = wait_bar(&bars[0], phase, abort_flag);
        if (!__syncthreads_and(ok)) break;
        if (tid == 0) {
            pending = false;
            tc_fence_after_sync();
            constexpr uint32_t id = idesc_bf16(128, 64, false, false);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint64_t d = smem_desc(sbase + L::KQ + (ks >> 2) * 16384 + (ks & 3) * 32, 16,
                                             1024, kSw128);
                mma_bf16(tmem, d, d, id, ks > 0);
            }
            mma_commit(&bars[1]);
        }
        ok = wait_bar(&bars[1], phase, abort_flag);
        phase ^= 1;
        if (!__syncthreads_and(ok)) break;
        tc_fence_after_sync();
        if (tid == 0 && next < o.total) pending = load(next);

        // rows of A and Att
        {
            const int r = tid & 63, R = r >> 4;
            const bool att = warp >= 2;
            const bool live = r < cr.valid;
            const double pr = psum[r];
            const float er = pexp[r] * (att ? a.scale : 1.f);
            const float lead = att ? a.scale : 1.f;
            float between = 1.f;  // whole blocks between column block I and row block R
            const int top = (r | 31) >> 4;  // blocks of this warp's last row
            // from the diagonal leftwards: I = R, R-1, ...
#pragma unroll
            for (int I = 3; I >= 0; --I) {
                if (I > top) {  // right of every row of this warp: zero
                    if (att) {
                        *reinterpret_cast<uint4*>(sm + L::IMG + kBlkAtt + sw128_off(r, 2 * I)) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4*>(sm + L::IMG + kBlkAtt + sw128_off(r, 2 * I + 1)) = make_uint4(0, 0, 0, 0);
                    }
                    continue;
                }
                float g[16];
                tmem_ld16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + 16 * I, g);
                tmem_wait_ld();
                const float off = er * between;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int c = 16 * I + j;
                    float f;
                    if (I < R) f = off * sbeta[c];
                    else f = lead * beta[c] * expf((float)(pr - psum[c]));
                    const bool in = live && (att ? c <= r : c < r);
                    g[j] = in ? g[j] * f : 0.f;  // a select: what is masked may be NaN
                }
                if (I < R) between *= btot[I];
                if (att) {
                    st_bf16x8(sm + L::IMG + kBlkAtt + sw128_off(r, 2 * I), g);
                    st_bf16x8(sm + L::IMG + kBlkAtt + sw128_off(r, 2 * I + 1), g + 8);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4*>(Am + r * LDA + 16 * I + j) =
                            make_float4(g[j], g[j + 1], g[j + 2], g[j + 3]);
                }
            }
        }
        tc_fence_before_sync();
        __syncthreads();
        // diagonal blocks: column c of block b by forward substitution
        if (warp < 2) {
            const int b = warp * 2 + (lane >> 4), c = lane & 15;
            float* blk = Am + (16 * b) * LDA + 16 * b;
            float x[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float y = r == c ? 1.f : 0.f;
#pragma unroll
                for (int k4 = 0; k4 < r; k4 += 4) {
                    const float4 w = lds4(blk + r * LDA + k4);
                    const float wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (k4 + e < r) y = fmaf(-wv[e], x[k4 + e], y);
                }
                x[r] = y;
            }
            __syncwarp();
#pragma unroll
            for (int r = 0; r < 16; ++r) blk[r * LDA + c] = x[r];
        }
        __syncthreads();
        // 16 -> 32: pair p of blocks, 64 threads, 4 columns of one row each
        {
            const int p = warp >> 1, t = tid & 63, r = t >> 2, c = (t & 3) * 4;
            float* lo = Am + (32 * p) * LDA + 32 * p;                 // T_00
            float* a10 = lo + 16 * LDA;                               // A_10
            float* t11 = a10 + 16;                                    // T_11
            float* scr = lo + 16;                                     // above the diagonal: scratch
            float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k4 = 0; k4 < 16; k4 += 4) {
                const float4 w = lds4(a10 + r * LDA + k4);
                const float wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 z = lds4(lo + (k4 + e) * LDA + c);
                    m[0] = fmaf(wv[e], z.x, m[0]);
                    m[1] = fmaf(wv[e], z.y, m[1]);
                    m[2] = fmaf(wv[e], z.z, m[2]);
                    m[3] = fmaf(wv[e], z.w, m[3]);
                }
            }
            *reinterpret_cast<float4*>(scr + r * LDA + c) = make_float4(m[0], m[1], m[2], m[3]);
            if (p == 0) named_bar(1, 64);
            else named_bar(2, 64);
            m[0] = m[1] = m[2] = m[3] = 0.f;
#pragma unroll
            for (int k4 = 0; k4 < 16; k4 += 4) {
                const float4 w = lds4(t11 + r * LDA + k4);
                const float wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 z = lds4(scr + (k4 + e) * LDA + c);
                    m[0] = fmaf(-wv[e], z.x, m[0]);
                    m[1] = fmaf(-wv[e], z.y, m[1]);
                    m[2] = fmaf(-wv[e], z.z, m[2]);
                    m[3] = fmaf(-wv[e], z.w, m[3]);
                }
            }
            *reinterpret_cast<float4*>(a10 + r * LDA + c) = make_float4(m[0], m[1], m[2], m[3]);
        }
        __syncthreads();
        // 32 -> 64: M = A_10 T_00 (above the diagonal), T_10 = -T_11 M.  The 16 x 16
        // blocks above T_00's and T_11's diagonals hold scratch and are skipped.
        {
            float m[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) m[e] = 0.f;
            const int c0 = 8 * warp;  // a warp: 8 columns, a lane per row
#pragma unroll 2
            for (int k4 = warp >= 2 ? 16 : 0; k4 < 32; k4 += 4) {
                const float4 w = lds4(Am + (32 + lane) * LDA + k4);
                const float wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 z0 = lds4(Am + (k4 + e) * LDA + c0), z1 = lds4(Am + (k4 + e) * LDA + c0 + 4);
                    m[0] = fmaf(wv[e], z0.x, m[0]); m[1] = fmaf(wv[e], z0.y, m[1]);
                    m[2] = fmaf(wv[e], z0.z, m[2]); m[3] = fmaf(wv[e], z0.w, m[3]);
                    m[4] = fmaf(wv[e], z1.x, m[4]); m[5] = fmaf(wv[e], z1.y, m[5]);
                    m[6] = fmaf(wv[e], z1.z, m[6]); m[7] = fmaf(wv[e], z1.w, m[7]);
                }
            }
            float* dst = Am + lane * LDA + 32 + c0;
            *reinterpret_cast<float4*>(dst) = make_float4(m[0], m[1], m[2], m[3]);
            *reinterpret_cast<float4*>(dst + 4) = make_float4(m[4], m[5], m[6], m[7]);
            __syncthreads();
            const int r0 = 8 * warp;  // a warp: 8 rows, a lane per column
#pragma unroll
            for (int e = 0; e < 8; ++e) m[e] = 0.f;
#pragma unroll 2
            for (int k4 = 0; k4 < (warp >= 2 ? 32 : 16); k4 += 4) {
                float z[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] = Am[(k4 + e) * LDA + 32 + lane];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 w = lds4(Am + (32 + r0 + j) * LDA + 32 + k4);
                    m[j] = fmaf(-w.x, z[0], fmaf(-w.y, z[1], fmaf(-w.z, z[2], fmaf(-w.w, z[3], m[j]))));
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) Am[(32 + r0 + j) * LDA + lane] = m[j];
        }
        __syncthreads();
        // T in two bf16 terms: a thread half a row
        {
            const int r = tid >> 1, half = tid & 1;
#pragma unroll
            for (int g8 = 0; g8 < 4; ++g8) {
                const int c = 32 * half + 8 * g8;
                uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
                if ((c >> 4) <= (r >> 4)) {
                    float x[8];
                    const float4 u = lds4(Am + r * LDA + c), w = lds4(Am + r * LDA + c + 4);
                    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
                    x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
                    split8(x, hi, lo);
                }
                *reinterpret_cast<uint4*>(sm + L::IMG + kBlkThi + sw128_off(r, c >> 3)) = hi;
                *reinterpret_cast<uint4*>(sm + L::IMG + kBlkTlo + sw128_off(r, c >> 3)) = lo;
            }
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            bulk_store(o.blk + (size_t)(n * a.H + h) * kBlkBytes, sm + L::IMG, kBlkBytes);
            bulk_commit_group();
        }
    }
    if (tid == 0) {
        if (pending) (void)mbar_wait(&bars[0], phase);  // after an abort: the load must land first
        bulk_wait_group_all();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (tid == 0 && *abort_flag) atomicOr(a.status + 1, 1u);
    if (warp == 0) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 64);
    }
}

template <int D>
cudaError_t launch_typed(const Args& a, cudaStream_t s)
{
    using L = Lay<D>;
    CUtensorMap mq, mk;
    if (!make_rows_map(&mq, a.q, a, a.Hk, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_rows_map(&mk, a.k, a, a.Hk, 64, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    int dev = 0, sms = 148;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(operands_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)L::BYTES);
    if (e != cudaSuccess) return e;
    OpArgs o;
    o.a = a;
    o.blk = a.blk;
    o.chunk_order = a.chunk_order;
    o.total = chunks(a) * a.H;
    if (o.total == 0) return cudaSuccess;
    const long long grid = o.total < 3LL * sms ? o.total : 3LL * sms;
    ProfScope ps(kGdrOperands, s);
    operands_kernel<D><<<(unsigned)grid, kThreads, L::BYTES, s>>>(mq, mk, o);
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

cudaError_t launch_operands_tc(const Args& a, cudaStream_t s)
{
    return a.D == 64 ? launch_typed<64>(a, s) : launch_typed<128>(a, s);
}

}  // namespace gdr
}  // namespace mdn
