// The gated delta rule on CUDA cores, in fp32: forward, and the three kernels
// of its backward pass (the formulas are in gdr_internal.cuh).
//
// The state is small (d x d) and its columns (rows, in the backward's last
// kernel) do not depend on one another, so a chain keeps it in registers for
// the whole sequence and walks the tokens.  A thread holds 4 columns and every
// eighth float4 of rows; the 8 lanes that share a column reduce by shuffles.
// One reduction per token is enough: with the state before the token,
//     o_t = scale (alpha S^T q + beta (k.q) vtilde),
// so S^T k and S^T q are summed together.  Bound by FMA issue: 3 d^2 per
// token and head (49,152 at d = 128, 384 cycles of an SM).
#include "gdr_internal.cuh"

namespace mdn {
namespace gdr {
namespace {

constexpr int TB = 16;   // tokens staged in shared memory at once
constexpr int RL = 8;    // lanes sharing a column (a row, in the token gradients)

__device__ __forceinline__ float dot4(const float4 a, const float4 b, float c)
{
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
// Sum over the RL lanes that share a column, in every lane.
__device__ __forceinline__ float lanes_sum(float x)
{
#pragma unroll
    for (int off = 1; off < RL; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// n token rows of width W of a [rows, heads, D] tensor as fp32 into dst[.][W]
// (zeros for tokens n .. TB-1); col0 is the first column.
template <typename T, int W, int D, int NT_>
__device__ __forceinline__ void stage(float (*dst)[W], const T* src, long long row0, int heads,
                                      int head, int col0, int n)
{
    for (int e = threadIdx.x; e < TB * W; e += NT_) {
        const int t = e / W, c = e % W;
        dst[t][c] = t < n ? ld_elem(src + ((size_t)(row0 + t) * heads + head) * D + col0 + c) : 0.f;
    }
}

// ---------------------------------------------------------------- forward
// One CTA: NC columns of one chain.
template <typename T, int D, int NC>
__global__ void __launch_bounds__(NC * 2) fwd_kernel(const Args a)
{
    constexpr int NTH = NC * 2, V = D / (4 * RL);  // float4 rows groups per thread
    __shared__ __align__(16) float ks[TB][D], qs[TB][D], vs[TB][NC];
    __shared__ float al[TB], be[TB], kq[TB];
    const Chain ch = chain_of(a, blockIdx.x / (D / NC));
    const int col0 = (blockIdx.x % (D / NC)) * NC;
    const int tid = threadIdx.x, rl = tid % RL, cg = tid / RL;  // 4 columns 4 cg ..
    float s[V * 4][4];
    const size_t sbase = (size_t)ch.state * D * D + col0 + cg * 4;
#pragma unroll
    for (int i = 0; i < V * 4; ++i) {
        const int r = (i / 4) * (4 * RL) + rl * 4 + i % 4;
        const float4 x = a.S0 ? *reinterpret_cast<const float4*>(a.S0 + sbase + (size_t)r * D)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        s[i][0] = x.x; s[i][1] = x.y; s[i][2] = x.z; s[i][3] = x.w;
    }
    for (int t0 = 0; t0 < ch.len; t0 += TB) {
        const int n = min(TB, ch.len - t0);
        const long long row = ch.row0 + t0;
        __syncthreads();
        stage<T, D, D, NTH>(ks, static_cast<const T*>(a.k), row, a.Hk, ch.hk, 0, n);
        stage<T, D, D, NTH>(qs, static_cast<const T*>(a.q), row, a.Hk, ch.hk, 0, n);
        stage<T, NC, D, NTH>(vs, static_cast<const T*>(a.v), row, a.H, ch.h, col0, n);
        if (tid < n) {
            al[tid] = expf(a.alpha_log[(row + tid) * a.H + ch.h]);
            be[tid] = a.beta[(row + tid) * a.H + ch.h];
        }
        __syncthreads();
        for (int t = tid / 8; t < TB; t += NTH / 8) {  // k.q of each token, 8 lanes a token
            float x = 0.f;
            for (int i = tid % 8; i < D; i += 8) x = fmaf(ks[t][i], qs[t][i], x);
            x = lanes_sum(x);
            if (tid % 8 == 0) kq[t] = x;
        }
        __syncthreads();
        for (int t = 0; t < n; ++t) {
            float pk[4] = {0.f, 0.f, 0.f, 0.f}, pq[4] = {0.f, 0.f, 0.f, 0.f};
            float kr[V * 4];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float4 k4 = *reinterpret_cast<const float4*>(&ks[t][i * (4 * RL) + rl * 4]);
                const float4 q4 = *reinterpret_cast<const float4*>(&qs[t][i * (4 * RL) + rl * 4]);
                kr[4 * i] = k4.x; kr[4 * i + 1] = k4.y; kr[4 * i + 2] = k4.z; kr[4 * i + 3] = k4.w;
                const float qr[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        pk[c] = fmaf(s[4 * i + e][c], kr[4 * i + e], pk[c]);
                        pq[c] = fmaf(s[4 * i + e][c], qr[e], pq[c]);
                    }
            }
            const float alpha = al[t], b = be[t];
            float x[4], ov[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[c] = vs[t][cg * 4 + c] - alpha * lanes_sum(pk[c]);
                ov[c] = a.scale * fmaf(alpha, lanes_sum(pq[c]), b * kq[t] * x[c]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float bx = b * x[c];
#pragma unroll
                for (int i = 0; i < V * 4; ++i) s[i][c] = fmaf(alpha, s[i][c], kr[i] * bx);
            }
            const size_t out = ((size_t)(row + t) * a.H + ch.h) * D + col0 + cg * 4;
            if (rl < 4) {
                float y = ov[0];
                y = rl == 1 ? ov[1] : rl == 2 ? ov[2] : rl == 3 ? ov[3] : y;
                st_elem(static_cast<T*>(a.o) + out + rl, y);
            } else if (a.vt) {
                float y = x[0];
                y = rl == 5 ? x[1] : rl == 6 ? x[2] : rl == 7 ? x[3] : y;
                st_elem(static_cast<T*>(a.vt) + out + rl - 4, y);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V * 4; ++i) {
        const int r = (i / 4) * (4 * RL) + rl * 4 + i % 4;
        *reinterpret_cast<float4*>(a.S_T + sbase + (size_t)r * D) =
            make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
    }
}

// ---------------------------------------------------------------- backward
// S entering each chunk, from the saved vtilde (no chain of products: the
// update of a token reads nothing of the state but its scale).
template <typename T, int D, int NC>
__global__ void __launch_bounds__(NC * 2) states_kernel(const Args a)
{
    constexpr int NTH = NC * 2, V = D / (4 * RL);
    __shared__ __align__(16) float ks[TB][D], vs[TB][NC];
    __shared__ float al[TB], be[TB];
    const Chain ch = chain_of(a, blockIdx.x / (D / NC));
    const int col0 = (blockIdx.x % (D / NC)) * NC;
    const int tid = threadIdx.x, rl = tid % RL, cg = tid / RL;
    float s[V * 4][4];
    const size_t sbase = (size_t)ch.state * D * D + col0 + cg * 4;
#pragma unroll
    for (int i = 0; i < V * 4; ++i) {
        const int r = (i / 4) * (4 * RL) + rl * 4 + i % 4;
        const float4 x = a.S0 ? *reinterpret_cast<const float4*>(a.S0 + sbase + (size_t)r * D)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        s[i][0] = x.x; s[i][1] = x.y; s[i][2] = x.z; s[i][3] = x.w;
    }
    for (int t0 = 0; t0 < ch.len; t0 += TB) {
        if (t0 % kChunk == 0) {
            float* dst = a.SS + ((size_t)(ch.chunk0 + t0 / kChunk) * a.H + ch.h) * D * D + col0 + cg * 4;
#pragma unroll
            for (int i = 0; i < V * 4; ++i) {
                const int r = (i / 4) * (4 * RL) + rl * 4 + i % 4;
                *reinterpret_cast<float4*>(dst + (size_t)r * D) =
                    make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
            }
        }
        const int n = min(TB, ch.len - t0);
        const long long row = ch.row0 + t0;
        __syncthreads();
        stage<T, D, D, NTH>(ks, static_cast<const T*>(a.k), row, a.Hk, ch.hk, 0, n);
        stage<T, NC, D, NTH>(vs, static_cast<const T*>(a.vt), row, a.H, ch.h, col0, n);
        if (tid < n) {
            al[tid] = expf(a.alpha_log[(row + tid) * a.H + ch.h]);
            be[tid] = a.beta[(row + tid) * a.H + ch.h];
        }
        __syncthreads();
        for (int t = 0; t < n; ++t) {
            const float alpha = al[t];
            float bx[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) bx[c] = be[t] * vs[t][cg * 4 + c];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float4 k4 = *reinterpret_cast<const float4*>(&ks[t][i * (4 * RL) + rl * 4]);
                const float kr[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        s[4 * i + e][c] = fmaf(alpha, s[4 * i + e][c], kr[e] * bx[c]);
            }
        }
    }
}

// The reverse chain: dv, the adjoint of S leaving each chunk, dS0.  As in the
// forward pass one reduction per token: with the adjoint G' from the later
// tokens, dv = beta (G'^T k + scale (q.k) do).
template <typename T, int D, int NC>
__global__ void __launch_bounds__(NC * 2) reverse_kernel(const Args a)
{
    constexpr int NTH = NC * 2, V = D / (4 * RL);
    __shared__ __align__(16) float ks[TB][D], qs[TB][D], os[TB][NC];
    __shared__ float al[TB], be[TB], kq[TB];
    const Chain ch = chain_of(a, blockIdx.x / (D / NC));
    const int col0 = (blockIdx.x % (D / NC)) * NC;
    const int tid = threadIdx.x, rl = tid % RL, cg = tid / RL;
    float g[V * 4][4];
    const size_t sbase = (size_t)ch.state * D * D + col0 + cg * 4;
#pragma unroll
    for (int i = 0; i < V * 4; ++i) {
        const int r = (i / 4) * (4 * RL) + rl * 4 + i % 4;
        const float4 x = a.dS_T ? *reinterpret_cast<const float4*>(a.dS_T + sbase + (size_t)r * D)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
        g[i][0] = x.x; g[i][1] = x.y; g[i][2] = x.z; g[i][3] = x.w;
    }
    for (int t0 = (ch.len - 1) / TB * TB; t0 >= 0 && ch.len > 0; t0 -= TB) {
        const int n = min(TB, ch.len - t0);
        if (t0 + n == ch.len || (t0 + TB) % kChunk == 0) {
            float* dst = a.GG + ((size_t)(ch.chunk0 + t0 / kChunk) * a.H + ch.h) * D * D + col0 + cg * 4;
#pragma unroll
            for (int i = 0; i < V * 4; ++i) {
                const int r = (i / 4) * (4 * RL) + rl * 4 + i % 4;
                *reinterpret_cast<float4*>(dst + (size_t)r * D) =
                    make_float4(g[i][0], g[i][1], g[i][2], g[i][3]);
            }
        }
        const long long row = ch.row0 + t0;
        __syncthreads();
        stage<T, D, D, NTH>(ks, static_cast<const T*>(a.k), row, a.Hk, ch.hk, 0, n);
        stage<T, D, D, NTH>(qs, static_cast<const T*>(a.q), row, a.Hk, ch.hk, 0, n);
        stage<T, NC, D, NTH>(os, static_cast<const T*>(a.d_o), row, a.H, ch.h, col0, n);
        if (tid < n) {
            al[tid] = expf(a.alpha_log[(row + tid) * a.H + ch.h]);
            be[tid] = a.beta[(row + tid) * a.H + ch.h];
        }
        __syncthreads();
        for (int t = tid / 8; t < TB; t += NTH / 8) {
            float x = 0.f;
            for (int i = tid % 8; i < D; i += 8) x = fmaf(ks[t][i], qs[t][i], x);
            x = lanes_sum(x);
            if (tid % 8 == 0) kq[t] = a.scale * x;
        }
        __syncthreads();
        for (int t = n - 1; t >= 0; --t) {
            float p[4] = {0.f, 0.f, 0.f, 0.f};
            float kr[V * 4];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float4 k4 = *reinterpret_cast<const float4*>(&ks[t][i * (4 * RL) + rl * 4]);
                kr[4 * i] = k4.x; kr[4 * i + 1] = k4.y; kr[4 * i + 2] = k4.z; kr[4 * i + 3] = k4.w;
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int c = 0; c < 4; ++c) p[c] = fmaf(g[4 * i + e][c], kr[4 * i + e], p[c]);
            }
            const float alpha = al[t];
            float dv[4], od[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float d = os[t][cg * 4 + c];
                dv[c] = be[t] * fmaf(kq[t], d, lanes_sum(p[c]));
                od[c] = a.scale * d;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float4 q4 = *reinterpret_cast<const float4*>(&qs[t][i * (4 * RL) + rl * 4]);
                const float qr[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        g[4 * i + e][c] = alpha * fmaf(-kr[4 * i + e], dv[c],
                                                       fmaf(qr[e], od[c], g[4 * i + e][c]));
            }
            if (rl < 4) {
                float y = dv[0];
                y = rl == 1 ? dv[1] : rl == 2 ? dv[2] : rl == 3 ? dv[3] : y;
                const size_t out = ((size_t)(row + t) * a.H + ch.h) * D + col0 + cg * 4 + rl;
                a.dvf[out] = y;
                st_elem(static_cast<T*>(a.dv) + out, y);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V * 4; ++i) {
        const int r = (i / 4) * (4 * RL) + rl * 4 + i % 4;
        *reinterpret_cast<float4*>(a.dS0 + sbase + (size_t)r * D) =
            make_float4(g[i][0], g[i][1], g[i][2], g[i][3]);
    }
}

// The token gradients of one chunk of one head, from the S entering it and
// the adjoint of the S leaving it: rows of S and of G are independent here, so
// a thread holds 4 rows and every eighth float4 of columns.  Forward over the
// tokens for dq and alpha S dv, backward for G vtilde.  dalpha_log follows
// from   dalpha_log_t = dalpha_log_{t+1} + q.dq - beta dbeta - alpha k.(S dv),
// started at the chunk's end with <G, S>, so that sums stay inside a chunk.
template <typename T, int D>
__global__ void __launch_bounds__(D * 2) token_grads_kernel(const Args a)
{
    constexpr int NTH = D * 2, V = D / (4 * RL), NW = NTH / 32;
    extern __shared__ __align__(16) float sh[];
    float (*c0)[D] = reinterpret_cast<float (*)[D]>(sh);               // do (forward), vtilde
    float (*c1)[D] = reinterpret_cast<float (*)[D]>(sh + TB * D);      // dv
    float (*c2)[D] = reinterpret_cast<float (*)[D]>(sh + 2 * TB * D);  // vtilde (forward), do
    float (*ks)[D] = reinterpret_cast<float (*)[D]>(sh + 3 * TB * D);
    float (*qs)[D] = reinterpret_cast<float (*)[D]>(sh + 4 * TB * D);
    float (*dks)[D] = reinterpret_cast<float (*)[D]>(sh + 5 * TB * D);  // [64] alpha S dv
    __shared__ float al[TB], be[TB], dd[TB];
    __shared__ float cc[kChunk][NW], bb[kChunk][NW];  // a warp's share of q.dq - k.(alpha S dv); dbeta
    __shared__ float ip[NW];
    const long long n = blockIdx.x / a.H;
    const int h = blockIdx.x % a.H, hk = h / (a.H / a.Hk);
    const ChunkRows cr = chunk_rows(a, n);
    if (cr.valid <= 0) return;
    const int tid = threadIdx.x, rl = tid % RL, rg = tid / RL, warp = tid / 32, lane = tid % 32;
    const int row4 = rg * 4;
    const size_t sbase = ((size_t)n * a.H + h) * D * D + (size_t)row4 * D;
    float s[4][V * 4];
    auto load = [&](const float* src) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float4 x = *reinterpret_cast<const float4*>(src + sbase + r * D + i * (4 * RL) + rl * 4);
                s[r][4 * i] = x.x; s[r][4 * i + 1] = x.y; s[r][4 * i + 2] = x.z; s[r][4 * i + 3] = x.w;
            }
    };
    auto stage_all = [&](int t0, int m, const T* x0, const T* x2) {
        const long long row = cr.row0 + t0;
        __syncthreads();
        stage<T, D, D, NTH>(c0, x0, row, a.H, h, 0, m);
        stage<float, D, D, NTH>(c1, a.dvf, row, a.H, h, 0, m);
        stage<T, D, D, NTH>(c2, x2, row, a.H, h, 0, m);
        stage<T, D, D, NTH>(ks, static_cast<const T*>(a.k), row, a.Hk, hk, 0, m);
        stage<T, D, D, NTH>(qs, static_cast<const T*>(a.q), row, a.Hk, hk, 0, m);
        if (tid < m) {
            al[tid] = expf(a.alpha_log[(row + tid) * a.H + h]);
            be[tid] = a.beta[(row + tid) * a.H + h];
        }
        __syncthreads();
        for (int t = tid / 8; t < TB; t += NTH / 8) {
            float x = 0.f;
            for (int i = tid % 8; i < D; i += 8) x = fmaf(c0[t][i], c2[t][i], x);
            x = lanes_sum(x);
            if (tid % 8 == 0) dd[t] = x;  // do . vtilde
        }
        __syncthreads();
    };
    const T* vt = static_cast<const T*>(a.vt);
    const T* dout = static_cast<const T*>(a.d_o);
    load(a.SS);
    for (int t0 = 0; t0 < cr.valid; t0 += TB) {
        const int m = min(TB, cr.valid - t0);
        stage_all(t0, m, dout, vt);
        for (int t = 0; t < m; ++t) {
            float po[4] = {0.f, 0.f, 0.f, 0.f}, pd[4] = {0.f, 0.f, 0.f, 0.f};
            const float alpha = al[t], b = be[t];
            float bk[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) bk[r] = b * ks[t][row4 + r];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = i * (4 * RL) + rl * 4;
                const float4 o4 = *reinterpret_cast<const float4*>(&c0[t][c]);
                const float4 d4 = *reinterpret_cast<const float4*>(&c1[t][c]);
                const float4 v4 = *reinterpret_cast<const float4*>(&c2[t][c]);
                const float vv[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float4 s4 = make_float4(s[r][4 * i], s[r][4 * i + 1], s[r][4 * i + 2], s[r][4 * i + 3]);
                    po[r] = dot4(s4, o4, po[r]);
                    pd[r] = dot4(s4, d4, pd[r]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[r][4 * i + e] = fmaf(alpha, s[r][4 * i + e], bk[r] * vv[e]);
                }
            }
            float share = 0.f;
            float dq[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                dq[r] = a.scale * fmaf(alpha, lanes_sum(po[r]), bk[r] * dd[t]);
                pd[r] = alpha * lanes_sum(pd[r]);
                share += qs[t][row4 + r] * dq[r] - ks[t][row4 + r] * pd[r];
            }
            const size_t tok = (size_t)(cr.row0 + t0 + t);
            if (rl < 4) {
                float y = dq[0], z = pd[0];
                y = rl == 1 ? dq[1] : rl == 2 ? dq[2] : rl == 3 ? dq[3] : y;
                z = rl == 1 ? pd[1] : rl == 2 ? pd[2] : rl == 3 ? pd[3] : z;
                dks[t0 + t][row4 + rl] = z;
                if (a.dqp) a.dqp[(tok * a.H + h) * D + row4 + rl] = y;
                else st_elem(static_cast<T*>(a.dq) + (tok * a.Hk + hk) * D + row4 + rl, y);
            }
            // the 4 row groups of the warp
            share += __shfl_xor_sync(0xffffffffu, share, 8);
            share += __shfl_xor_sync(0xffffffffu, share, 16);
            if (lane == 0) cc[t0 + t][warp] = share;
        }
    }
    // <G, S> at the chunk's end, then G
    {
        float x = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float4 g4 = *reinterpret_cast<const float4*>(a.GG + sbase + r * D + i * (4 * RL) + rl * 4);
                x = dot4(g4, make_float4(s[r][4 * i], s[r][4 * i + 1], s[r][4 * i + 2], s[r][4 * i + 3]), x);
            }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        if (lane == 0) ip[warp] = x;
    }
    load(a.GG);
    for (int t0 = (cr.valid - 1) / TB * TB; t0 >= 0; t0 -= TB) {
        const int m = min(TB, cr.valid - t0);
        stage_all(t0, m, vt, dout);
        for (int t = m - 1; t >= 0; --t) {
            float p[4] = {0.f, 0.f, 0.f, 0.f};
            const float alpha = al[t], b = be[t];
            float sq[4], kr[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                sq[r] = a.scale * qs[t][row4 + r];
                kr[r] = ks[t][row4 + r];
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = i * (4 * RL) + rl * 4;
                const float4 v4 = *reinterpret_cast<const float4*>(&c0[t][c]);
                const float4 d4 = *reinterpret_cast<const float4*>(&c1[t][c]);
                const float4 o4 = *reinterpret_cast<const float4*>(&c2[t][c]);
                const float vv[4] = {v4.x, v4.y, v4.z, v4.w}, dv[4] = {d4.x, d4.y, d4.z, d4.w};
                const float od[4] = {o4.x, o4.y, o4.z, o4.w};
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float& g = s[r][4 * i + e];
                        p[r] = fmaf(g, vv[e], p[r]);
                        g = alpha * fmaf(-kr[r], dv[e], fmaf(sq[r], od[e], g));
                    }
            }
            float share = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                p[r] = fmaf(sq[r], dd[t], lanes_sum(p[r]));
                share = fmaf(kr[r], p[r], share);
            }
            const size_t tok = (size_t)(cr.row0 + t0 + t);
            if (rl < 4) {
                float z = p[0];
                z = rl == 1 ? p[1] : rl == 2 ? p[2] : rl == 3 ? p[3] : z;
                const float y = fmaf(b, z, -dks[t0 + t][row4 + rl]);
                if (a.dkp) a.dkp[(tok * a.H + h) * D + row4 + rl] = y;
                else st_elem(static_cast<T*>(a.dk) + (tok * a.Hk + hk) * D + row4 + rl, y);
            }
            share += __shfl_xor_sync(0xffffffffu, share, 8);
            share += __shfl_xor_sync(0xffffffffu, share, 16);
            if (lane == 0) bb[t0 + t][warp] = share;
        }
    }
    __syncthreads();
    // warp 0: dbeta, and dalpha_log as a suffix sum over the chunk's tokens
    if (warp == 0) {
        float c[2], b[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            c[e] = b[e] = 0.f;
            if (t < cr.valid) {
                const size_t at = (size_t)(cr.row0 + t) * a.H + h;
                for (int w = 0; w < NW; ++w) {
                    c[e] += cc[t][w];
                    b[e] += bb[t][w];
                }
                c[e] = fmaf(-a.beta[at], b[e], c[e]);
                a.dbeta[at] = b[e];
            }
        }
        float end = 0.f;
        for (int w = 0; w < NW; ++w) end += ip[w];
        float x = c[0] + c[1];  // inclusive suffix sum over lanes
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float y = __shfl_down_sync(0xffffffffu, x, off);
            if (lane + off < 32) x += y;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            if (t < cr.valid) {
                float y = (e == 0 ? x : x - c[0]) + end;
                // nothing enters a sequence's first token from no state: its decay has no effect
                if (t == 0 && cr.first && !a.S0) y = 0.f;
                a.dalpha_log[(size_t)(cr.row0 + t) * a.H + h] = y;
            }
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(256) fold_kernel(const Args a, long long total)
{
    const long long e = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;  // of [rows, Hk, D]
    if (e >= total) return;
    const int rep = a.H / a.Hk;
    const long long rk = e / D;  // row * Hk + hk; its value heads are rk * rep ..
    if (a.cu_s && rk / a.Hk >= a.cu_s[a.B]) return;  // rows behind the last sequence
    const size_t src = (size_t)rk * rep * D + e % D;
    float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
    for (int r = 0; r < rep; ++r) {
        const float4 p = *reinterpret_cast<const float4*>(a.dqp + src + (size_t)r * D);
        const float4 u = *reinterpret_cast<const float4*>(a.dkp + src + (size_t)r * D);
        x[0] += p.x; x[1] += p.y; x[2] += p.z; x[3] += p.w;
        y[0] += u.x; y[1] += u.y; y[2] += u.z; y[3] += u.w;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        st_elem(static_cast<T*>(a.dq) + e + c, x[c]);
        st_elem(static_cast<T*>(a.dk) + e + c, y[c]);
    }
}

int sm_count()
{
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

// Columns per CTA: 32 while the narrow CTAs fit on the SMs four at a time
// (the shortest walk per token), else the whole head (a token's q and k are
// then staged once).
template <typename T, int D>
cudaError_t fwd_typed(const Args& a, cudaStream_t s)
{
    const long long n = chains(a);
    ProfScope ps(kGdrFwdSimt, s);
    if (n * (D / 32) <= 4LL * sm_count())
        fwd_kernel<T, D, 32><<<(unsigned)(n * (D / 32)), 64, 0, s>>>(a);
    else
        fwd_kernel<T, D, D><<<(unsigned)n, 2 * D, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t bwd_typed(const Args& a, cudaStream_t s)
{
    const long long n = chains(a);
    const bool narrow = n * (D / 32) <= 4LL * sm_count();
    cudaError_t e;
    {
        ProfScope ps(kGdrBwdStates, s);
        if (narrow) states_kernel<T, D, 32><<<(unsigned)(n * (D / 32)), 64, 0, s>>>(a);
        else states_kernel<T, D, D><<<(unsigned)n, 2 * D, 0, s>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    {
        ProfScope ps(kGdrBwdChain, s);
        if (narrow) reverse_kernel<T, D, 32><<<(unsigned)(n * (D / 32)), 64, 0, s>>>(a);
        else reverse_kernel<T, D, D><<<(unsigned)n, 2 * D, 0, s>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    constexpr int shm = (5 * TB + kChunk) * D * (int)sizeof(float);
    if ((e = cudaFuncSetAttribute(token_grads_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  shm)) != cudaSuccess)
        return e;
    const long long blocks = chunks(a) * a.H;
    if (blocks == 0) return cudaSuccess;
    ProfScope ps(kGdrBwdGrads, s);
    token_grads_kernel<T, D><<<(unsigned)blocks, 2 * D, shm, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fold_heads(const Args& a, mdn_dtype dt, cudaStream_t s)
{
    const long long total = rows(a) * a.Hk * a.D;
    const unsigned blocks = (unsigned)((total / 4 + 255) / 256);
    if (blocks == 0) return cudaSuccess;
    ProfScope ps(kGdrFold, s);
    if (dt == MDN_F32) {
        if (a.D == 64) fold_kernel<float, 64><<<blocks, 256, 0, s>>>(a, total);
        else fold_kernel<float, 128><<<blocks, 256, 0, s>>>(a, total);
    } else {
        if (a.D == 64) fold_kernel<__nv_bfloat16, 64><<<blocks, 256, 0, s>>>(a, total);
        else fold_kernel<__nv_bfloat16, 128><<<blocks, 256, 0, s>>>(a, total);
    }
    return cudaGetLastError();
}

cudaError_t launch_fwd_simt(const Args& a, mdn_dtype dt, cudaStream_t s)
{
    if (dt == MDN_F32) return a.D == 64 ? fwd_typed<float, 64>(a, s) : fwd_typed<float, 128>(a, s);
    return a.D == 64 ? fwd_typed<__nv_bfloat16, 64>(a, s) : fwd_typed<__nv_bfloat16, 128>(a, s);
}

cudaError_t launch_bwd_simt(const Args& a, mdn_dtype dt, cudaStream_t s)
{
    if (dt == MDN_F32) return a.D == 64 ? bwd_typed<float, 64>(a, s) : bwd_typed<float, 128>(a, s);
    return a.D == 64 ? bwd_typed<__nv_bfloat16, 64>(a, s) : bwd_typed<__nv_bfloat16, 128>(a, s);
}

}  // namespace gdr
}  // namespace mdn
