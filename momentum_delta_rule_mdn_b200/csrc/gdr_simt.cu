// The gated delta rule on CUDA cores, in fp32: forward, and the three kernels
// of its backward pass (the formulas are in gdr_internal.cuh).
//
// The state is small (d x d) and its columns (rows, in the backward's last
// kernel) do not depend on one another, so a chain keeps it in registers for
// the whole sequence and walks the tokens.  A thread holds 1 or 4 columns and every
// eighth float4 of rows; the 8 lanes that share a column reduce by shuffles.
// One reduction per token is enough: with the state before the token,
//     o_t = scale (alpha S^T q + beta (k.q) vtilde),
// so S^T k and S^T q are summed together.  Bound by FMA issue: 3 d^2 per
// token and head (49,152 at d = 128, 384 cycles of an SM).
#include "gdr_internal.cuh"

namespace mdn {
namespace gdr {
namespace {

constexpr int TB = 16;   // tokens staged in shared memory at once (two such buffers)
constexpr int kGradTokens = 8;  // the same of the token gradients' kernel (more tensors a token)
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

// n token rows of width W of a [rows, heads, D] tensor into dst[TB][W], as stored
// and asynchronously, 16 bytes at a time (zeros for tokens n .. TB-1); col0 is the
// first column.  Complete after stage_commit and stage_wait.
template <typename T, int TB, int W, int D, int NT_>
__device__ __forceinline__ void stage(T* dst, const T* src, long long row0, int heads, int head,
                                      int col0, int n)
{
    constexpr int P = W * (int)sizeof(T) / 16;  // pieces of a row
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    for (int e = threadIdx.x; e < TB * P; e += NT_) {
        const int t = e / P, c = e % P;
        const T* from = src + ((size_t)(row0 + (t < n ? t : 0)) * heads + head) * D + col0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + e * 16),
                     "l"(reinterpret_cast<const char*>(from) + c * 16), "r"(t < n ? 16 : 0)
                     : "memory");
    }
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits for all but the newest group.
__device__ __forceinline__ void stage_wait() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

__device__ __forceinline__ float4 get4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 get4(const __nv_bfloat16* p)
{
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}

// Two buffers of TB token rows: `rows` elements of T (and `frows` floats) per token.
template <typename T, int TB_, int ROWS>
struct Buffers {
    T* base;
    __device__ __forceinline__ T* at(int k, int off) const { return base + ((size_t)(k & 1) * ROWS + off) * TB_; }
};

// Dot products of two staged rows, 8 lanes a token.
template <typename T, int TB, int D, int NT_>
__device__ __forceinline__ void dots(float* out, const T* x, const T* y, float f)
{
    for (int t = threadIdx.x / 8; t < TB; t += NT_ / 8) {
        float s = 0.f;
#pragma unroll
        for (int i = (threadIdx.x % 8) * 4; i < D; i += 32) s = dot4(get4(x + t * D + i), get4(y + t * D + i), s);
        s = lanes_sum(s);
        if (threadIdx.x % 8 == 0) out[t] = f * s;
    }
}

// A thread's part of a state: CPT columns from c0, rows 4 rl .. of every 32.
template <int D, int CPT>
struct Part {
    static constexpr int V = D / (4 * RL), R = 4 * V;  // rows of a thread
    float s[R][CPT];
    __device__ static __forceinline__ int row(int i, int rl) { return (i / 4) * (4 * RL) + rl * 4 + i % 4; }
    __device__ __forceinline__ void load(const float* src, int rl)  // src: the first column, or null (zeros)
    {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if constexpr (CPT == 4) {
                const float4 x = src ? *reinterpret_cast<const float4*>(src + (size_t)row(i, rl) * D)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                s[i][0] = x.x; s[i][1] = x.y; s[i][2] = x.z; s[i][3] = x.w;
            } else {
#pragma unroll
                for (int c = 0; c < CPT; ++c) s[i][c] = src ? src[(size_t)row(i, rl) * D + c] : 0.f;
            }
        }
    }
    __device__ __forceinline__ void store(float* dst, int rl) const
    {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if constexpr (CPT == 4) {
                *reinterpret_cast<float4*>(dst + (size_t)row(i, rl) * D) =
                    make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
            } else {
#pragma unroll
                for (int c = 0; c < CPT; ++c) dst[(size_t)row(i, rl) * D + c] = s[i][c];
            }
        }
    }
};
template <int V, typename T>
__device__ __forceinline__ void get_rows(float (&x)[4 * V], const T* row, int rl)
{
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float4 k4 = get4(row + i * (4 * RL) + rl * 4);
        x[4 * i] = k4.x; x[4 * i + 1] = k4.y; x[4 * i + 2] = k4.z; x[4 * i + 3] = k4.w;
    }
}
template <int CPT, typename T>
__device__ __forceinline__ void get_cols(float (&x)[CPT], const T* p)
{
    if constexpr (CPT == 4) {
        const float4 v = get4(p);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
#pragma unroll
        for (int c = 0; c < CPT; ++c) x[c] = ld_elem(p + c);
    }
}
// x[rl], with x in registers.
template <int CPT>
__device__ __forceinline__ float pick(const float (&x)[CPT], int rl)
{
    float y = x[0];
#pragma unroll
    for (int c = 1; c < CPT; ++c) y = rl == c ? x[c] : y;
    return y;
}

// ---------------------------------------------------------------- forward
// One CTA: NC columns of one chain, CPT of them per thread.
template <typename T, int D, int NC, int CPT>
__global__ void __launch_bounds__(NC / CPT * RL) fwd_kernel(const Args a)
{
    constexpr int NTH = NC / CPT * RL, V = D / (4 * RL), R = 4 * V;
    extern __shared__ __align__(16) uint8_t shm[];
    const Buffers<T, TB, 2 * D + NC> buf{reinterpret_cast<T*>(shm)};  // k, q, v
    __shared__ float al[TB], be[TB], kq[TB];
    const Chain ch = chain_of(a, blockIdx.x / (D / NC));
    const int col0 = (blockIdx.x % (D / NC)) * NC;
    const int tid = threadIdx.x, rl = tid % RL, c0 = tid / RL * CPT;
    const size_t sbase = (size_t)ch.state * D * D + col0 + c0;
    Part<D, CPT> st;
    st.load(a.S0 ? a.S0 + sbase : nullptr, rl);
    float ga = 0.f, gb = 0.f;  // gates of token tid of the block being fetched
    auto fetch = [&](int t0, int k) {
        const int n = min(TB, ch.len - t0);
        const long long row = ch.row0 + t0;
        if (n > 0) {
            stage<T, TB, D, D, NTH>(buf.at(k, 0), static_cast<const T*>(a.k), row, a.Hk, ch.hk, 0, n);
            stage<T, TB, D, D, NTH>(buf.at(k, D), static_cast<const T*>(a.q), row, a.Hk, ch.hk, 0, n);
            stage<T, TB, NC, D, NTH>(buf.at(k, 2 * D), static_cast<const T*>(a.v), row, a.H, ch.h, col0, n);
            if (tid < n) {
                ga = a.alpha_log[(row + tid) * a.H + ch.h];
                gb = a.beta[(row + tid) * a.H + ch.h];
            }
        }
        stage_commit();
    };
    fetch(0, 0);
    for (int t0 = 0, k = 0; t0 < ch.len; t0 += TB, ++k) {
        const int n = min(TB, ch.len - t0);
        const T* ks = buf.at(k, 0);
        const T* qs = buf.at(k, D);
        const T* vs = buf.at(k, 2 * D);
        __syncthreads();  // the other buffer, al, be, kq are free
        if (tid < TB) {
            al[tid] = expf(ga);
            be[tid] = gb;
        }
        fetch(t0 + TB, k + 1);
        stage_wait();
        __syncthreads();
        dots<T, TB, D, NTH>(kq, ks, qs, 1.f);
        __syncthreads();
        const size_t out0 = ((size_t)(ch.row0 + t0) * a.H + ch.h) * D + col0 + c0;
        // lane c of a column group stores o of its column c, lane CPT + c vtilde
        T* dst = rl < CPT ? static_cast<T*>(a.o) + out0 + rl
                          : a.vt && rl < 2 * CPT ? static_cast<T*>(a.vt) + out0 + rl - CPT : nullptr;
#pragma unroll 2
        for (int t = 0; t < n; ++t) {
            float pk[CPT], pq[CPT], kr[R], qr[R], v[CPT];
#pragma unroll
            for (int c = 0; c < CPT; ++c) pk[c] = pq[c] = 0.f;
            get_rows<V>(kr, ks + t * D, rl);
            get_rows<V>(qr, qs + t * D, rl);
            get_cols<CPT>(v, vs + t * NC + c0);
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
                    pk[c] = fmaf(st.s[i][c], kr[i], pk[c]);
                    pq[c] = fmaf(st.s[i][c], qr[i], pq[c]);
                }
            const float alpha = al[t], b = be[t];
            float x[CPT], ov[CPT];
#pragma unroll
            for (int c = 0; c < CPT; ++c) {
                x[c] = v[c] - alpha * lanes_sum(pk[c]);
                ov[c] = a.scale * fmaf(alpha, lanes_sum(pq[c]), b * kq[t] * x[c]);
            }
#pragma unroll
            for (int c = 0; c < CPT; ++c) {
                const float bx = b * x[c];
#pragma unroll
                for (int i = 0; i < R; ++i) st.s[i][c] = fmaf(alpha, st.s[i][c], kr[i] * bx);
            }
            if (dst) st_elem(dst + (size_t)t * a.H * D, rl < CPT ? pick<CPT>(ov, rl) : pick<CPT>(x, rl - CPT));
        }
    }
    st.store(a.S_T + sbase, rl);
}

// ---------------------------------------------------------------- backward
// S entering each chunk, from the saved vtilde (no chain of products: the
// update of a token reads nothing of the state but its scale).
template <typename T, int D, int NC, int CPT>
__global__ void __launch_bounds__(NC / CPT * RL) states_kernel(const Args a)
{
    constexpr int NTH = NC / CPT * RL, V = D / (4 * RL), R = 4 * V;
    extern __shared__ __align__(16) uint8_t shm[];
    const Buffers<T, TB, D + NC> buf{reinterpret_cast<T*>(shm)};  // k, vtilde
    __shared__ float al[TB], be[TB];
    const Chain ch = chain_of(a, blockIdx.x / (D / NC));
    const int col0 = (blockIdx.x % (D / NC)) * NC;
    const int tid = threadIdx.x, rl = tid % RL, c0 = tid / RL * CPT;
    const size_t sbase = (size_t)ch.state * D * D + col0 + c0;
    Part<D, CPT> st;
    st.load(a.S0 ? a.S0 + sbase : nullptr, rl);
    float ga = 0.f, gb = 0.f;
    auto fetch = [&](int t0, int k) {
        const int n = min(TB, ch.len - t0);
        const long long row = ch.row0 + t0;
        if (n > 0) {
            stage<T, TB, D, D, NTH>(buf.at(k, 0), static_cast<const T*>(a.k), row, a.Hk, ch.hk, 0, n);
            stage<T, TB, NC, D, NTH>(buf.at(k, D), static_cast<const T*>(a.vt), row, a.H, ch.h, col0, n);
            if (tid < n) {
                ga = a.alpha_log[(row + tid) * a.H + ch.h];
                gb = a.beta[(row + tid) * a.H + ch.h];
            }
        }
        stage_commit();
    };
    fetch(0, 0);
    for (int t0 = 0, k = 0; t0 < ch.len; t0 += TB, ++k) {
        if (t0 % kChunk == 0)
            st.store(a.SS + ((size_t)(ch.chunk0 + t0 / kChunk) * a.H + ch.h) * D * D + col0 + c0, rl);
        const int n = min(TB, ch.len - t0);
        const T* ks = buf.at(k, 0);
        const T* vs = buf.at(k, D);
        __syncthreads();
        if (tid < TB) {
            al[tid] = expf(ga);
            be[tid] = gb;
        }
        fetch(t0 + TB, k + 1);
        stage_wait();
        __syncthreads();
#pragma unroll 4
        for (int t = 0; t < n; ++t) {
            const float alpha = al[t], b = be[t];
            float kr[R], v[CPT];
            get_rows<V>(kr, ks + t * D, rl);
            get_cols<CPT>(v, vs + t * NC + c0);
#pragma unroll
            for (int c = 0; c < CPT; ++c) {
                const float bx = b * v[c];
#pragma unroll
                for (int i = 0; i < R; ++i) st.s[i][c] = fmaf(alpha, st.s[i][c], kr[i] * bx);
            }
        }
    }
}

// The reverse chain: dv, the adjoint of S leaving each chunk, dS0.  As in the
// forward pass one reduction per token: with the adjoint G' from the later
// tokens, dv = beta (G'^T k + scale (q.k) do).
template <typename T, int D, int NC, int CPT>
__global__ void __launch_bounds__(NC / CPT * RL) reverse_kernel(const Args a)
{
    constexpr int NTH = NC / CPT * RL, V = D / (4 * RL), R = 4 * V;
    extern __shared__ __align__(16) uint8_t shm[];
    const Buffers<T, TB, 2 * D + NC> buf{reinterpret_cast<T*>(shm)};  // k, q, do
    __shared__ float al[TB], be[TB], kq[TB];
    const Chain ch = chain_of(a, blockIdx.x / (D / NC));
    const int col0 = (blockIdx.x % (D / NC)) * NC;
    const int tid = threadIdx.x, rl = tid % RL, c0 = tid / RL * CPT;
    const size_t sbase = (size_t)ch.state * D * D + col0 + c0;
    Part<D, CPT> g;
    g.load(a.dS_T ? a.dS_T + sbase : nullptr, rl);
    float ga = 0.f, gb = 0.f;
    auto fetch = [&](int t0, int k) {
        if (t0 >= 0) {
            const int n = min(TB, ch.len - t0);
            const long long row = ch.row0 + t0;
            stage<T, TB, D, D, NTH>(buf.at(k, 0), static_cast<const T*>(a.k), row, a.Hk, ch.hk, 0, n);
            stage<T, TB, D, D, NTH>(buf.at(k, D), static_cast<const T*>(a.q), row, a.Hk, ch.hk, 0, n);
            stage<T, TB, NC, D, NTH>(buf.at(k, 2 * D), static_cast<const T*>(a.d_o), row, a.H, ch.h, col0, n);
            if (tid < n) {
                ga = a.alpha_log[(row + tid) * a.H + ch.h];
                gb = a.beta[(row + tid) * a.H + ch.h];
            }
        }
        stage_commit();
    };
    const int top = ch.len > 0 ? (ch.len - 1) / TB * TB : -TB;
    fetch(top, 0);
    for (int t0 = top, k = 0; t0 >= 0; t0 -= TB, ++k) {
        const int n = min(TB, ch.len - t0);
        if (t0 + n == ch.len || (t0 + TB) % kChunk == 0)
            g.store(a.GG + ((size_t)(ch.chunk0 + t0 / kChunk) * a.H + ch.h) * D * D + col0 + c0, rl);
        const T* ks = buf.at(k, 0);
        const T* qs = buf.at(k, D);
        const T* os = buf.at(k, 2 * D);
        __syncthreads();
        if (tid < TB) {
            al[tid] = expf(ga);
            be[tid] = gb;
        }
        fetch(t0 - TB, k + 1);
        stage_wait();
        __syncthreads();
        dots<T, TB, D, NTH>(kq, ks, qs, a.scale);
        __syncthreads();
        const size_t out0 = ((size_t)(ch.row0 + t0) * a.H + ch.h) * D + col0 + c0 + rl;
#pragma unroll 2
        for (int t = n - 1; t >= 0; --t) {
            float p[CPT], kr[R], qr[R], o[CPT];
#pragma unroll
            for (int c = 0; c < CPT; ++c) p[c] = 0.f;
            get_rows<V>(kr, ks + t * D, rl);
            get_rows<V>(qr, qs + t * D, rl);
            get_cols<CPT>(o, os + t * NC + c0);
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int c = 0; c < CPT; ++c) p[c] = fmaf(g.s[i][c], kr[i], p[c]);
            const float alpha = al[t];
            float dv[CPT];
#pragma unroll
            for (int c = 0; c < CPT; ++c) {
                const float od = a.scale * o[c];
                dv[c] = be[t] * fmaf(kq[t], o[c], lanes_sum(p[c]));
#pragma unroll
                for (int i = 0; i < R; ++i)
                    g.s[i][c] = alpha * fmaf(-kr[i], dv[c], fmaf(qr[i], od, g.s[i][c]));
            }
            if (rl < CPT) {
                const float y = pick<CPT>(dv, rl);
                a.dvf[out0 + (size_t)t * a.H * D] = y;
                st_elem(static_cast<T*>(a.dv) + out0 + (size_t)t * a.H * D, y);
            }
        }
    }
    g.store(a.dS0 + sbase, rl);
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
    constexpr int NTH = D * 2, V = D / (4 * RL), NW = NTH / 32, TB = kGradTokens;
    extern __shared__ __align__(16) uint8_t shm[];
    float (*dks)[D] = reinterpret_cast<float (*)[D]>(shm);       // [64] alpha S dv
    const Buffers<float, TB, D> fbuf{reinterpret_cast<float*>(shm + kChunk * D * 4)};  // dv
    const Buffers<T, TB, 4 * D> buf{reinterpret_cast<T*>(shm + (kChunk + 2 * TB) * D * 4)};  // do, vtilde, k, q
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
    // blocks of tokens: forward over the chunk, then backward; k counts them
    float ga = 0.f, gb = 0.f;
    auto fetch = [&](int t0, int k) {
        const int m = min(TB, cr.valid - t0);
        const long long row = cr.row0 + t0;
        if (t0 >= 0 && m > 0) {
            stage<float, TB, D, D, NTH>(fbuf.at(k, 0), a.dvf, row, a.H, h, 0, m);
            stage<T, TB, D, D, NTH>(buf.at(k, 0), static_cast<const T*>(a.d_o), row, a.H, h, 0, m);
            stage<T, TB, D, D, NTH>(buf.at(k, D), static_cast<const T*>(a.vt), row, a.H, h, 0, m);
            stage<T, TB, D, D, NTH>(buf.at(k, 2 * D), static_cast<const T*>(a.k), row, a.Hk, hk, 0, m);
            stage<T, TB, D, D, NTH>(buf.at(k, 3 * D), static_cast<const T*>(a.q), row, a.Hk, hk, 0, m);
            if (tid < m) {
                ga = a.alpha_log[(row + tid) * a.H + h];
                gb = a.beta[(row + tid) * a.H + h];
            }
        }
        stage_commit();
    };
    auto turn = [&](int next, int k) {  // block k has landed, block k + 1 is on its way
        __syncthreads();
        if (tid < TB) {
            al[tid] = expf(ga);
            be[tid] = gb;
        }
        fetch(next, k + 1);
        stage_wait();
        __syncthreads();
        dots<T, TB, D, NTH>(dd, buf.at(k, 0), buf.at(k, D), 1.f);  // do . vtilde
        __syncthreads();
    };
    const int top = (cr.valid - 1) / TB * TB;
    int blk = 0;
    fetch(0, 0);
    load(a.SS);
    for (int t0 = 0; t0 < cr.valid; t0 += TB, ++blk) {
        const int m = min(TB, cr.valid - t0);
        turn(t0 + TB < cr.valid ? t0 + TB : top, blk);
        const float* c1 = fbuf.at(blk, 0);
        const T* c0 = buf.at(blk, 0);
        const T* c2 = buf.at(blk, D);
        const T* ks = buf.at(blk, 2 * D);
        const T* qs = buf.at(blk, 3 * D);
        for (int t = 0; t < m; ++t) {
            float po[4] = {0.f, 0.f, 0.f, 0.f}, pd[4] = {0.f, 0.f, 0.f, 0.f};
            const float alpha = al[t], b = be[t];
            const float4 k4 = get4(ks + t * D + row4), q4 = get4(qs + t * D + row4);
            const float kr[4] = {k4.x, k4.y, k4.z, k4.w}, qr[4] = {q4.x, q4.y, q4.z, q4.w};
            const float bk[4] = {b * k4.x, b * k4.y, b * k4.z, b * k4.w};
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = i * (4 * RL) + rl * 4;
                const float4 o4 = get4(c0 + t * D + c), d4 = get4(c1 + t * D + c), v4 = get4(c2 + t * D + c);
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
                share += qr[r] * dq[r] - kr[r] * pd[r];
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
    for (int t0 = top; t0 >= 0; t0 -= TB, ++blk) {
        const int m = min(TB, cr.valid - t0);
        turn(t0 - TB, blk);
        const float* c1 = fbuf.at(blk, 0);
        const T* c2 = buf.at(blk, 0);
        const T* c0 = buf.at(blk, D);
        const T* ks = buf.at(blk, 2 * D);
        const T* qs = buf.at(blk, 3 * D);
        for (int t = m - 1; t >= 0; --t) {
            float p[4] = {0.f, 0.f, 0.f, 0.f};
            const float alpha = al[t], b = be[t];
            const float4 k4 = get4(ks + t * D + row4), q4 = get4(qs + t * D + row4);
            const float kr[4] = {k4.x, k4.y, k4.z, k4.w};
            const float sq[4] = {a.scale * q4.x, a.scale * q4.y, a.scale * q4.z, a.scale * q4.w};
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = i * (4 * RL) + rl * 4;
                const float4 v4 = get4(c0 + t * D + c), d4 = get4(c1 + t * D + c), o4 = get4(c2 + t * D + c);
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

// One kernel with its dynamic shared memory.
template <typename K>
cudaError_t run(K kernel, long long blocks, int threads, size_t shm, cudaStream_t s, const Args& a)
{
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shm);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)blocks, threads, shm, s>>>(a);
    return cudaGetLastError();
}

// Columns per CTA and thread.  Few chains: 32 columns a CTA and one a thread, so
// that a token costs a warp few instructions (with one warp per scheduler each
// takes five to six cycles, whatever it does: four columns a thread took 0.94 us a
// token at d = 64, one 0.20 us); while those CTAs are at most two per SM.  More: the whole head a CTA and
// four columns a thread, which reads each staged k and q once for four columns.
template <typename T, int D>
cudaError_t fwd_typed(const Args& a, cudaStream_t s)
{
    const long long n = chains(a);
    ProfScope ps(kGdrFwdSimt, s);
    if (n * (D / 32) <= 2LL * sm_count())
        return run(fwd_kernel<T, D, 32, 1>, n * (D / 32), 32 * RL, 2 * TB * (2 * D + 32) * sizeof(T), s, a);
    return run(fwd_kernel<T, D, D, 4>, n, 2 * D, 2 * TB * 3 * D * sizeof(T), s, a);
}

template <typename T, int D>
cudaError_t bwd_typed(const Args& a, cudaStream_t s)
{
    const long long n = chains(a);
    const bool narrow = n * (D / 32) <= 2LL * sm_count();
    cudaError_t e;
    {
        ProfScope ps(kGdrBwdStates, s);
        e = narrow ? run(states_kernel<T, D, 32, 1>, n * (D / 32), 32 * RL, 2 * TB * (D + 32) * sizeof(T), s, a)
                   : run(states_kernel<T, D, D, 4>, n, 2 * D, 2 * TB * 2 * D * sizeof(T), s, a);
        if (e != cudaSuccess) return e;
    }
    {
        ProfScope ps(kGdrBwdChain, s);
        e = narrow ? run(reverse_kernel<T, D, 32, 1>, n * (D / 32), 32 * RL, 2 * TB * (2 * D + 32) * sizeof(T), s, a)
                   : run(reverse_kernel<T, D, D, 4>, n, 2 * D, 2 * TB * 3 * D * sizeof(T), s, a);
        if (e != cudaSuccess) return e;
    }
    const long long blocks = chunks(a) * a.H;
    if (blocks == 0) return cudaSuccess;
    ProfScope ps(kGdrBwdGrads, s);
    return run(token_grads_kernel<T, D>, blocks, 2 * D,
               (kChunk + 2 * kGradTokens) * D * sizeof(float) + 2 * kGradTokens * 4 * D * sizeof(T), s, a);
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
