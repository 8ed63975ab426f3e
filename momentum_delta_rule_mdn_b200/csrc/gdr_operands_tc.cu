// The chunk operands of the gated delta rule on sm_100a (formulas and layout in
// gdr_tc.cuh): one CTA of 128 threads per chunk and head at a time, three CTAs
// per SM, so that one CTA's dependent phases run under the others'.
//
//   1  [K; Q] by TMA; G = [K; Q] K^T on tcgen05 (M 128, N 64, K = d): exact
//      products of the inputs, fp32 sums; the next chunk's load follows at once
//   2  TMEM lane r is row r of A (lanes 0..63) or of Att (lanes 64..127).  Warp w < 2
//      writes rows 32 w .. of A to shared memory in fp32 and, alone, inverts
//      its two 16 x 16 diagonal blocks (a lane per column, forward substitution
//      with x in registers) and joins them, T_10 = -T_11 A_10 T_00; warps 2 and 3
//      write Att to the block image and scan the next chunk's gates meanwhile
//   3  the join of the two 32 x 32 halves, by all four warps, in fp32
//   4  T rounded to two bf16 terms into the image; one bulk store
//
// Bound by the latency of these phases (about 1.2k cycles of issue per chunk
// and SM); three CTAs per SM is what shared memory admits.
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
    static constexpr uint32_t BYTES = MISC + 16;
    static_assert(BARS % 8 == 0 && AM % 16 == 0, "alignment");
    static_assert(CTAS * (BYTES + 1024) <= 233472, "CTAs per SM");
};

struct OpArgs {
    Args a;
    uint8_t* blk;
    const int* chunk_order;
    int total;  // chunk-heads
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

// acc (2 rows x 4 columns) += sign * X[rows] Y[:, cols] over k in [k0, k1): X rows at x, x + LDA,
// Y rows at y; both fp32 with leading dimension LDA.
template <bool NEG>
__device__ __forceinline__ void tile_mm(float (&acc)[2][4], const float* x, const float* y, int k0, int k1)
{
#pragma unroll 4
    for (int k = k0; k < k1; k += 4) {
        const float4 x0 = lds4(x + k), x1 = lds4(x + LDA + k);
        const float xa[4] = {x0.x, x0.y, x0.z, x0.w}, xb[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 v = lds4(y + (k + e) * LDA);
            const float a0 = NEG ? -xa[e] : xa[e], a1 = NEG ? -xb[e] : xb[e];
            acc[0][0] = fmaf(a0, v.x, acc[0][0]); acc[0][1] = fmaf(a0, v.y, acc[0][1]);
            acc[0][2] = fmaf(a0, v.z, acc[0][2]); acc[0][3] = fmaf(a0, v.w, acc[0][3]);
            acc[1][0] = fmaf(a1, v.x, acc[1][0]); acc[1][1] = fmaf(a1, v.y, acc[1][1]);
            acc[1][2] = fmaf(a1, v.z, acc[1][2]); acc[1][3] = fmaf(a1, v.w, acc[1][3]);
        }
    }
}
__device__ __forceinline__ void tile_st(float* dst, const float (&acc)[2][4])
{
#pragma unroll
    for (int j = 0; j < 2; ++j)
        *reinterpret_cast<float4*>(dst + j * LDA) = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
}
__device__ __forceinline__ void tile_zero(float (&acc)[2][4])
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
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BARS);  // [0] load, [1] product
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC + 4);
    float* Am = reinterpret_cast<float*>(sm + L::AM);
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
    // Chunks with no tokens (a packed call's bound on its chunks) end the work order.
    const int step = gridDim.x;
    int i = blockIdx.x;
    bool more = false, pending = false;
    Item x, nx;
    if (i < o.total) {
        x = item(o, i);
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
    bool next = more && i + step < o.total;
    if (next) {
        nx = item(o, i + step);
        next = nx.valid > 0;
        if (next && warp == 2) load_gates(nx);
    }
    __syncthreads();
    for (int k = 0; more; ++k) {
        const GateVec gv = vec(k);
        const float* bt = btot(k);
        bool ok = true;
        if (warp == 0) {
            ok = wait_bar(&bars[0], k & 1, abort_flag);
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
            if (lane == 0) bulk_wait_group_read<0>();  // the last image has left
            __syncwarp();
        }
        ok = wait_bar(&bars[1], k & 1, abort_flag) && ok;
        if (!__syncthreads_and(ok)) break;
        tc_fence_after_sync();
        if (tid == 96) {
            pending = next;
            if (next) load(nx);
        }
        // ---- rows of A and Att, the diagonal 32 x 32 halves of T
        {
            const int r = tid & 63, R = r >> 4;
            const bool att = warp >= 2, live = r < x.valid;
            const uint32_t t0 = tmem + (static_cast<uint32_t>(warp * 32) << 16);
            const float ph = gv.at(kP, r), pl = gv.at(kPlo, r);
            // forward: column i carries beta_i; backward: row r of A carries beta_r
            const float lead = att ? a.scale : BWD ? gv.at(kBeta, r) : 1.f;
            float fd[16];  // factors of this row's diagonal block
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float4 p4 = gv.get4(kP, 4 * R + g), l4 = gv.get4(kPlo, 4 * R + g);
                const float4 b4 = gv.get4(kBeta, 4 * R + g);
                const float pv[4] = {p4.x, p4.y, p4.z, p4.w}, lv[4] = {l4.x, l4.y, l4.z, l4.w};
                const float bv[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    fd[4 * g + e] = (BWD ? lead : lead * bv[e]) * __expf((ph - pv[e]) + (pl - lv[e]));
            }
            const float ep = expf(ph);
            float off = lead * fmaf(ep, pl, ep);  // exp(p_r), then times the whole blocks between
            const int last = r & 15;              // columns of the diagonal block that count
            // row block R of lanes 16..31 is the warp's right-most column block
#pragma unroll
            for (int I = 3; I >= 0; --I) {
                if (I > ((warp & 1) ? 3 : 1)) continue;  // right of every row of this warp
                float g[16];
                tmem_ld16(t0 + 16 * I, g);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 s4 = gv.get4(kSbeta, 4 * I + q);
                    const float sv[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = 4 * q + e;
                        const float f = I == R ? fd[j] : off * sv[e];
                        const bool in = live && (I < R || (I == R && (att ? j <= last : j < last)));
                        g[j] = in ? g[j] * f : 0.f;  // a select: what is masked may be NaN
                    }
                }
                if (I < R) off *= bt[I];
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
            const int rr = 2 * (lane >> 2), cc = 4 * (lane & 3);
            float acc[2][4];
            tile_zero(acc);
            tile_mm<false>(acc, lo + (16 + rr) * LDA, lo + cc, 0, 16);
            tile_st(lo + rr * LDA + 16 + cc, acc);
            __syncwarp();
            tile_zero(acc);
            tile_mm<true>(acc, lo + (16 + rr) * LDA + 16, lo + 16 + cc, 0, 16);
            tile_st(lo + (16 + rr) * LDA + cc, acc);
        } else if (warp == 2 && next) {
            scan_gates<BWD>(vec(k + 1), btot(k + 1), rec_of(nx), a.scale, ga, gb, lane);
        }
        const bool next2 = next && i + 2 * step < o.total;
        Item nx2 = nx;
        bool n2 = false;
        if (next2) {
            nx2 = item(o, i + 2 * step);
            n2 = nx2.valid > 0;
            if (n2 && warp == 2) load_gates(nx2);
        }
        __syncthreads();
        // ---- the two halves joined: M = A_10 T_00 (above the diagonal), T_10 = -T_11 M.
        // A warp takes 16 x 16 of the result; the 16 x 16 blocks above T_00's and T_11's own
        // diagonals (scratch, mathematically zero) are skipped.
        {
            const int u = warp >> 1, v = warp & 1, rr = 2 * (lane >> 2), cc = 4 * (lane & 3);
            float acc[2][4];
            tile_zero(acc);  // rows 16 v .., columns 16 u ..
            tile_mm<false>(acc, Am + (32 + 16 * v + rr) * LDA, Am + 16 * u + cc, 16 * u, 32);
            tile_st(Am + (16 * v + rr) * LDA + 32 + 16 * u + cc, acc);
            __syncthreads();
            tile_zero(acc);  // rows 16 u .., columns 16 v ..
            tile_mm<true>(acc, Am + (32 + 16 * u + rr) * LDA + 32, Am + 32 + 16 * v + cc, 0, 16 * (u + 1));
            tile_st(Am + (32 + 16 * u + rr) * LDA + 16 * v + cc, acc);
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
        }
        i += step;
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
    if (tid == 0) bulk_wait_group_all();
    tc_fence_before_sync();
    __syncthreads();
    if (tid == 0 && *abort_flag) atomicOr(a.status + 1, 1u);
    if (warp == 0) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 64);
    }
}

template <int D, bool BWD>
cudaError_t launch_typed(const Args& a, cudaStream_t s)
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

cudaError_t launch_operands_tc(const Args& a, cudaStream_t s, bool bwd)
{
    if (bwd) return launch_typed<128, true>(a, s);
    return a.D == 64 ? launch_typed<64, false>(a, s) : launch_typed<128, false>(a, s);
}

}  // namespace gdr
}  // namespace mdn
