// One decode token of the gated delta rule (formulas in gdr_internal.cuh).
//
// Bound by HBM: every state element is read once and written once.  A block
// owns one head and NC of its columns; a thread 4 adjacent columns (float4)
// and D / RG rows.  With the state before the token,
//     vtilde = v - alpha S^T k,   o = scale (alpha S^T q + beta (k.q) vtilde),
// so both column sums come from one pass over the registers and one
// reduction, and the stores of the new state follow the only barrier.  4096 heads of
// d 128: 88 us, 554 MB at 6.3 TB/s; 16 heads: 4.5 us (kernel alone, state in L2), 6 us replayed
// in a graph from cold caches, a launch and its latency.
#include "gdr_internal.cuh"

namespace mdn {
namespace gdr {
namespace {

template <typename T, int D, int NC>
__global__ void __launch_bounds__(256)
step_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
            const float* __restrict__ alpha_log, const float* __restrict__ beta, float scale,
            const float* S, float* S_out, T* __restrict__ o, T* __restrict__ vt, int rep)
{
    constexpr int CG = NC / 4, RG = 256 / CG, RP = D / RG, PARTS = D / NC;
    static_assert(RP >= 1 && CG <= 32, "shape");
    __shared__ float2 kq[D];              // k, q of a row
    __shared__ float2 red[8][NC];         // S^T k, S^T q: a warp's share
    __shared__ float dots[8];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long bh = blockIdx.x / PARTS, bk = bh / rep;  // value head, its key head
    const int col0 = (blockIdx.x % PARTS) * NC;
    const int cg = tid % CG, rg = tid / CG;
    const size_t base = (size_t)bh * D * D + col0 + cg * 4;
    float4 s4[RP];
#pragma unroll
    for (int e = 0; e < RP; ++e)
        s4[e] = __ldcs(reinterpret_cast<const float4*>(S + base + (size_t)(rg * RP + e) * D));
    const float alpha = expf(alpha_log[bh]), be = beta[bh];
    float d = 0.f;
    if (tid < D) {
        const float2 x = make_float2(ld_elem(k + (size_t)bk * D + tid), ld_elem(q + (size_t)bk * D + tid));
        kq[tid] = x;
        d = x.x * x.y;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    if (lane == 0) dots[warp] = d;
    float vj[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) vj[c] = ld_elem(v + (size_t)bh * D + col0 + cg * 4 + c);
    __syncthreads();
    float2 p[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) p[c] = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < RP; ++e) {
        const float2 x = kq[rg * RP + e];
        const float sv[4] = {s4[e].x, s4[e].y, s4[e].z, s4[e].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            p[c].x = fmaf(sv[c], x.x, p[c].x);
            p[c].y = fmaf(sv[c], x.y, p[c].y);
        }
    }
#pragma unroll
    for (int off = CG; off < 32; off <<= 1)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            p[c].x += __shfl_xor_sync(0xffffffffu, p[c].x, off);
            p[c].y += __shfl_xor_sync(0xffffffffu, p[c].y, off);
        }
    if (lane < CG) {
#pragma unroll
        for (int c = 0; c < 4; ++c) red[warp][cg * 4 + c] = p[c];
    }
    __syncthreads();
    float bx[4], x[4], pq[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {  // every thread sums its own columns: no second barrier
        float sk = 0.f, sq = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const float2 y = red[w][cg * 4 + c];
            sk += y.x;
            sq += y.y;
        }
        x[c] = vj[c] - alpha * sk;
        bx[c] = be * x[c];
        pq[c] = sq;
    }
#pragma unroll
    for (int e = 0; e < RP; ++e) {
        const float kv = kq[rg * RP + e].x;
        const float4 y = make_float4(fmaf(alpha, s4[e].x, kv * bx[0]), fmaf(alpha, s4[e].y, kv * bx[1]),
                                     fmaf(alpha, s4[e].z, kv * bx[2]), fmaf(alpha, s4[e].w, kv * bx[3]));
        __stcs(reinterpret_cast<float4*>(S_out + base + (size_t)(rg * RP + e) * D), y);
    }
    if (rg == 0) {
        float dot = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) dot += dots[w];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const size_t at = (size_t)bh * D + col0 + cg * 4 + c;
            st_elem(o + at, scale * fmaf(alpha, pq[c], dot * bx[c]));
            if (vt) st_elem(vt + at, x[c]);
        }
    }
}

template <typename T, int D>
cudaError_t step_typed(const void* q, const void* k, const void* v, const float* alpha_log,
                       const float* beta, float scale, const float* S, float* S_out, int B, int Hk,
                       int H, void* o, void* vt, cudaStream_t s)
{
    const long long heads = (long long)B * H;
    int dev = 0, sms = 148;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    ProfScope ps(kGdrStep, s);
    const T* qq = static_cast<const T*>(q);
    const T* kk = static_cast<const T*>(k);
    const T* vv = static_cast<const T*>(v);
    T* oo = static_cast<T*>(o);
    T* tt = static_cast<T*>(vt);
    const int rep = H / Hk;
    // the widest column split that still gives every SM two blocks
    if (heads * (D / 64) >= 2LL * sms)
        step_kernel<T, D, 64><<<(unsigned)(heads * (D / 64)), 256, 0, s>>>(
            qq, kk, vv, alpha_log, beta, scale, S, S_out, oo, tt, rep);
    else if (heads * (D / 32) >= 2LL * sms)
        step_kernel<T, D, 32><<<(unsigned)(heads * (D / 32)), 256, 0, s>>>(
            qq, kk, vv, alpha_log, beta, scale, S, S_out, oo, tt, rep);
    else
        step_kernel<T, D, 16><<<(unsigned)(heads * (D / 16)), 256, 0, s>>>(
            qq, kk, vv, alpha_log, beta, scale, S, S_out, oo, tt, rep);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_step(const void* q, const void* k, const void* v, mdn_dtype dt,
                        const float* alpha_log, const float* beta, float scale, const float* S,
                        float* S_out, int B, int Hk, int H, int D, void* o, void* vt,
                        cudaStream_t s)
{
    if (dt == MDN_F32)
        return D == 64 ? step_typed<float, 64>(q, k, v, alpha_log, beta, scale, S, S_out, B, Hk, H, o, vt, s)
                       : step_typed<float, 128>(q, k, v, alpha_log, beta, scale, S, S_out, B, Hk, H, o, vt, s);
    return D == 64 ? step_typed<__nv_bfloat16, 64>(q, k, v, alpha_log, beta, scale, S, S_out, B, Hk, H, o, vt, s)
                   : step_typed<__nv_bfloat16, 128>(q, k, v, alpha_log, beta, scale, S, S_out, B, Hk, H, o, vt, s);
}

}  // namespace gdr
}  // namespace mdn
