// The gated delta rule on CUDA cores, in fp32: forward, and the three kernels
// of its backward pass (the formulas are in gdr_internal.cuh).
//
// The state is small (d x d) and its columns (rows, in the backward's last
// kernel) do not depend on one another, so a chain keeps it in registers for
// the whole sequence and walks the tokens.  A thread holds 1 or 4 columns and every
// eighth float4 of rows; the 8 lanes that share a column reduce by shuffles.
// One reduction per token is enough: with the state before the token,
//     o_t = scale (alpha S^T q + beta (k.q) vtilde),
// so S^T k and S^T q are summed together; few chains share one among four tokens.
// Many chains are bound by FMA issue: 3 d^2 per token and head (49,152 at d = 128,
// 384 cycles of an SM); few by the latency of a token.
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

// Sums of 8 values over 8 lanes: lane rl returns the sum of value rl (7 shuffles; 24 if
// every lane formed every sum).
__device__ __forceinline__ float lanes_sum8(const float (&x)[8], int rl)
{
    float y[4], z[2];
    const bool b4 = rl & 4, b2 = rl & 2, b1 = rl & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = (b4 ? x[i + 4] : x[i]) + __shfl_xor_sync(0xffffffffu, b4 ? x[i] : x[i + 4], 4);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        z[i] = (b2 ? y[i + 2] : y[i]) + __shfl_xor_sync(0xffffffffu, b2 ? y[i] : y[i + 2], 2);
    return (b1 ? z[1] : z[0]) + __shfl_xor_sync(0xffffffffu, b1 ? z[0] : z[1], 1);
}
// The same of 4 values: lane rl returns value rl % 4 (4 shuffles).
__device__ __forceinline__ float lanes_sum4(const float (&x)[4], int rl)
{
    const bool b2 = rl & 2, b1 = rl & 1;
    float z[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        z[i] = (b2 ? x[i + 2] : x[i]) + __shfl_xor_sync(0xffffffffu, b2 ? x[i] : x[i + 2], 2);
    const float s = (b1 ? z[1] : z[0]) + __shfl_xor_sync(0xffffffffu, b1 ? z[0] : z[1], 1);
    return s + __shfl_xor_sync(0xffffffffu, s, 4);
}
// Lane i's value of s into x[i], in every lane of the 8.
template <int N>
__device__ __forceinline__ void spread(float (&x)[N], float s)
{
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __shfl_sync(0xffffffffu, s, i, 8);
}
__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
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

// ---------------------------------------------------------------- few chains
// With few chains a token's latency is the time, and most of it is the reduction.  So
// GT = 4 tokens share one: their products with the state before all four are summed
// together, and the three updates between are scalars per column, from the dot products
// of the four tokens with one another (16 per four tokens, the same for every column).
constexpr int GT = 4;
constexpr int kFew = 16;  // columns of a CTA (32: 0.19 us a token at d 64, 8: 0.18, 16: 0.17)

// Dot products inside every group of GT staged tokens, 8 lanes each: m[group][j][i] is
// x_j . y_i for i <= j (REV: or, forward, for i >= j) and x_j . x_i on the other side.
// Forward x = k, y = q; reverse x = q, y = k, and the other side is y_j . y_i.
template <typename T, int TB, int D, int NT_, bool REV>
__device__ __forceinline__ void grams(float (*m)[GT][GT], const T* ks, const T* qs)
{
    for (int e = threadIdx.x / 8; e < TB / GT * GT * GT; e += NT_ / 8) {
        const int g = e / (GT * GT), j = e / GT % GT, i = e % GT;
        const bool kq = REV ? i <= j : i >= j;
        // forward: k_j . q_i, else k_j . k_i; reverse: q_j . k_i, else k_j . k_i
        const T* x = (REV && kq ? qs : ks) + (g * GT + j) * D;
        const T* y = (!REV && kq ? qs : ks) + (g * GT + i) * D;
        float s = 0.f;
#pragma unroll
        for (int c = (threadIdx.x % 8) * 4; c < D; c += 32) s = dot4(get4(x + c), get4(y + c), s);
        s = lanes_sum(s);
        if (threadIdx.x % 8 == 0) m[g][j][i] = s;
    }
}

// Forward: with S the state before the group, u_i = S^T k_i and w_i = S^T q_i; token j
// turns every later u_i into alpha_j u_i + beta_j (k_j . k_i) vtilde_j, and w likewise.
template <typename T, int D, int NC>
__global__ void __launch_bounds__(NC * RL) fwd_few_kernel(const Args a)
{
    constexpr int NTH = NC * RL, V = D / (4 * RL), R = 4 * V;
    extern __shared__ __align__(16) uint8_t shm[];
    const Buffers<T, TB, 2 * D + NC> buf{reinterpret_cast<T*>(shm)};  // k, q, v
    __shared__ __align__(16) float al[TB], be[TB], gram[TB / GT][GT][GT];
    const Chain ch = chain_of(a, blockIdx.x / (D / NC));
    const int col0 = (blockIdx.x % (D / NC)) * NC;
    const int tid = threadIdx.x, rl = tid % RL, c0 = tid / RL;
    const size_t sbase = (size_t)ch.state * D * D + col0 + c0;
    Part<D, 1> st;
    st.load(a.S0 ? a.S0 + sbase : nullptr, rl);
    T* const dst0 = static_cast<T*>(rl < GT ? a.o : a.vt);
    const size_t hop = (size_t)GT * a.H * D;
    float ga = 0.f, gb = 0.f;  // gates of token tid of the block being fetched
    auto fetch = [&](int t0, int k) {
        const int n = min(TB, ch.len - t0);
        const long long row = ch.row0 + t0;
        if (n > 0) {
            stage<T, TB, D, D, NTH>(buf.at(k, 0), static_cast<const T*>(a.k), row, a.Hk, ch.hk, 0, n);
            stage<T, TB, D, D, NTH>(buf.at(k, D), static_cast<const T*>(a.q), row, a.Hk, ch.hk, 0, n);
            stage<T, TB, NC, D, NTH>(buf.at(k, 2 * D), static_cast<const T*>(a.v), row, a.H, ch.h, col0, n);
            const bool in = tid < n;  // behind the sequence: no decay, no update
            ga = in ? a.alpha_log[(row + tid) * a.H + ch.h] : 0.f;
            gb = in ? a.beta[(row + tid) * a.H + ch.h] : 0.f;
        }
        stage_commit();
    };
    fetch(0, 0);
    for (int t0 = 0, k = 0; t0 < ch.len; t0 += TB, ++k) {
        const int n = min(TB, ch.len - t0);
        const T* ks = buf.at(k, 0);
        const T* qs = buf.at(k, D);
        const T* vs = buf.at(k, 2 * D);
        __syncthreads();  // the other buffer, al, be, gram are free
        if (tid < TB) {
            al[tid] = expf(ga);
            be[tid] = gb;
        }
        fetch(t0 + TB, k + 1);
        stage_wait();
        __syncthreads();
        grams<T, TB, D, NTH, false>(gram, ks, qs);
        __syncthreads();
        // lane j stores o of token j of a group, lane GT + j vtilde
        T* dst = dst0;
        if (dst) dst += ((size_t)(ch.row0 + t0 + rl % GT) * a.H + ch.h) * D + col0 + c0;
#pragma unroll 1
        for (int t = 0; t < n; t += GT) {
            float kr[GT][R], x[2 * GT], v[GT];
#pragma unroll
            for (int j = 0; j < GT; ++j) {
                float qr[R];
                get_rows<V>(kr[j], ks + (t + j) * D, rl);
                get_rows<V>(qr, qs + (t + j) * D, rl);
                v[j] = ld_elem(vs + (t + j) * NC + c0);
                x[j] = x[GT + j] = 0.f;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    x[j] = fmaf(st.s[i][0], kr[j][i], x[j]);
                    x[GT + j] = fmaf(st.s[i][0], qr[i], x[GT + j]);
                }
            }
            const float4 a4 = get4(al + t), b4 = get4(be + t);
            const float av[GT] = {a4.x, a4.y, a4.z, a4.w}, bv[GT] = {b4.x, b4.y, b4.z, b4.w};
            spread(x, lanes_sum8(x, rl));
            float c[GT];
#pragma unroll
            for (int j = 0; j < GT; ++j) {
                const float4 m4 = get4(gram[t / GT][j]);
                const float m[GT] = {m4.x, m4.y, m4.z, m4.w};
                const float y = fmaf(-av[j], x[j], v[j]);
                c[j] = t + j < n ? bv[j] * y : 0.f;
                x[j] = y;
#pragma unroll
                for (int i = j + 1; i < GT; ++i) x[i] = fmaf(av[j], x[i], c[j] * gram[t / GT][i][j]);
#pragma unroll
                for (int i = 0; i < GT; ++i)
                    x[GT + i] = i < j ? x[GT + i] : fmaf(av[j], x[GT + i], c[j] * m[i]);
            }
            float after = 1.f;  // decay of the tokens behind j
#pragma unroll
            for (int j = GT - 1; j >= 0; --j) {
                c[j] *= after;
                after *= av[j];
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float s = st.s[i][0] * after;
#pragma unroll
                for (int j = 0; j < GT; ++j) s = fmaf(kr[j][i], c[j], s);
                st.s[i][0] = s;
            }
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < GT; ++i) y = rl % GT == i ? (rl < GT ? a.scale * x[GT + i] : x[i]) : y;
            if (dst && t + rl % GT < n) st_elem(dst, y);
            if (dst) dst += hop;
        }
    }
    st.store(a.S_T + sbase, rl);
}

// ---------------------------------------------------------------- forward
// One CTA: the D columns of one chain, CPT of them per thread.
template <typename T, int D>
__global__ void __launch_bounds__(D / 4 * RL) fwd_kernel(const Args a)
{
    constexpr int NC = D, CPT = 4, NTH = NC / CPT * RL, V = D / (4 * RL), R = 4 * V;
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
template <typename T, int D>
__global__ void __launch_bounds__(D / 4 * RL) states_kernel(const Args a)
{
    constexpr int NC = D, CPT = 4, NTH = NC / CPT * RL, V = D / (4 * RL), R = 4 * V;
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
template <typename T, int D>
__global__ void __launch_bounds__(D / 4 * RL) reverse_kernel(const Args a)
{
    constexpr int NC = D, CPT = 4, NTH = NC / CPT * RL, V = D / (4 * RL), R = 4 * V;
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

// Few chains: the two kernels above side by side (neither reads the other's results),
// GT tokens at a time, one column a thread.
template <typename T, int D, int NC>
__device__ __forceinline__ void states_few(const Args& a, int block, uint8_t* shm, float* al, float* be)
{
    constexpr int NTH = NC * RL, V = D / (4 * RL), R = 4 * V;
    const Buffers<T, TB, D + NC> buf{reinterpret_cast<T*>(shm)};  // k, vtilde
    const Chain ch = chain_of(a, block / (D / NC));
    const int col0 = (block % (D / NC)) * NC;
    const int tid = threadIdx.x, rl = tid % RL, c0 = tid / RL;
    const size_t sbase = (size_t)ch.state * D * D + col0 + c0;
    Part<D, 1> st;
    st.load(a.S0 ? a.S0 + sbase : nullptr, rl);
    float ga = 0.f, gb = 0.f;
    auto fetch = [&](int t0, int k) {
        const int n = min(TB, ch.len - t0);
        const long long row = ch.row0 + t0;
        if (n > 0) {
            stage<T, TB, D, D, NTH>(buf.at(k, 0), static_cast<const T*>(a.k), row, a.Hk, ch.hk, 0, n);
            stage<T, TB, NC, D, NTH>(buf.at(k, D), static_cast<const T*>(a.vt), row, a.H, ch.h, col0, n);
            const bool in = tid < n;
            ga = in ? a.alpha_log[(row + tid) * a.H + ch.h] : 0.f;
            gb = in ? a.beta[(row + tid) * a.H + ch.h] : 0.f;
        }
        stage_commit();
    };
    fetch(0, 0);
    for (int t0 = 0, k = 0; t0 < ch.len; t0 += TB, ++k) {
        if (t0 % kChunk == 0)
            st.store(a.SS + ((size_t)(ch.chunk0 + t0 / kChunk) * a.H + ch.h) * D * D + col0 + c0, rl);
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
        // all TB tokens: those behind the sequence are zero rows without decay
#pragma unroll 1
        for (int t = 0; t < TB; t += GT) {
            const float4 a4 = get4(al + t), b4 = get4(be + t);
            const float av[GT] = {a4.x, a4.y, a4.z, a4.w}, bv[GT] = {b4.x, b4.y, b4.z, b4.w};
            float kr[GT][R], c[GT], after = 1.f;
#pragma unroll
            for (int j = GT - 1; j >= 0; --j) {
                get_rows<V>(kr[j], ks + (t + j) * D, rl);
                c[j] = bv[j] * ld_elem(vs + (t + j) * NC + c0) * after;
                after *= av[j];
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float s = st.s[i][0] * after;
#pragma unroll
                for (int j = 0; j < GT; ++j) s = fmaf(kr[j][i], c[j], s);
                st.s[i][0] = s;
            }
        }
    }
}

// With G' the adjoint behind the group, u_i = G'^T k_i; token j, from the last, gives
// dv_j = beta_j (u_j + scale (q_j . k_j) do_j) and turns every earlier u_i into
// alpha_j (u_i + scale (q_j . k_i) do_j - (k_j . k_i) dv_j).
template <typename T, int D, int NC>
__device__ __forceinline__ void reverse_few(const Args& a, int block, uint8_t* shm, float* al, float* be,
                                            float (*gram)[GT][GT])
{
    constexpr int NTH = NC * RL, V = D / (4 * RL), R = 4 * V;
    const Buffers<T, TB, 2 * D + NC> buf{reinterpret_cast<T*>(shm)};  // k, q, do
    const Chain ch = chain_of(a, block / (D / NC));
    const int col0 = (block % (D / NC)) * NC;
    const int tid = threadIdx.x, rl = tid % RL, c0 = tid / RL;
    const size_t sbase = (size_t)ch.state * D * D + col0 + c0;
    Part<D, 1> g;
    g.load(a.dS_T ? a.dS_T + sbase : nullptr, rl);
    float ga = 0.f, gb = 0.f;
    auto fetch = [&](int t0, int k) {
        if (t0 >= 0) {
            const int n = min(TB, ch.len - t0);
            const long long row = ch.row0 + t0;
            stage<T, TB, D, D, NTH>(buf.at(k, 0), static_cast<const T*>(a.k), row, a.Hk, ch.hk, 0, n);
            stage<T, TB, D, D, NTH>(buf.at(k, D), static_cast<const T*>(a.q), row, a.Hk, ch.hk, 0, n);
            stage<T, TB, NC, D, NTH>(buf.at(k, 2 * D), static_cast<const T*>(a.d_o), row, a.H, ch.h, col0, n);
            const bool in = tid < n;
            ga = in ? a.alpha_log[(row + tid) * a.H + ch.h] : 0.f;
            gb = in ? a.beta[(row + tid) * a.H + ch.h] : 0.f;
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
        grams<T, TB, D, NTH, true>(gram, ks, qs);
        __syncthreads();
        const size_t out0 = ((size_t)(ch.row0 + t0) * a.H + ch.h) * D + col0 + c0;
#pragma unroll 1
        for (int t = (n - 1) / GT * GT; t >= 0; t -= GT) {
            float kr[GT][R], u[GT], h[GT], dv[GT];
#pragma unroll
            for (int j = 0; j < GT; ++j) {
                get_rows<V>(kr[j], ks + (t + j) * D, rl);
                h[j] = a.scale * ld_elem(os + (t + j) * NC + c0);
                u[j] = 0.f;
#pragma unroll
                for (int i = 0; i < R; ++i) u[j] = fmaf(g.s[i][0], kr[j][i], u[j]);
            }
            const float4 a4 = get4(al + t), b4 = get4(be + t);
            const float av[GT] = {a4.x, a4.y, a4.z, a4.w}, bv[GT] = {b4.x, b4.y, b4.z, b4.w};
            spread(u, lanes_sum4(u, rl));
#pragma unroll
            for (int j = GT - 1; j >= 0; --j) {
                const float4 m4 = get4(gram[t / GT][j]);
                const float m[GT] = {m4.x, m4.y, m4.z, m4.w};
                dv[j] = t + j < n ? bv[j] * fmaf(h[j], m[j], u[j]) : 0.f;
#pragma unroll
                for (int i = 0; i < j; ++i)
                    u[i] = av[j] * fmaf(-dv[j], gram[t / GT][i][j], fmaf(h[j], m[i], u[i]));
            }
            {
                const int j = rl % GT;
                float y = 0.f;
#pragma unroll
                for (int i = 0; i < GT; ++i) y = j == i ? dv[i] : y;
                if (rl < GT && t + j < n) {
                    const size_t at = out0 + (size_t)(t + j) * a.H * D;
                    a.dvf[at] = y;
                    st_elem(static_cast<T*>(a.dv) + at, y);
                }
            }
            float decay = 1.f;  // of the tokens up to j
#pragma unroll
            for (int j = 0; j < GT; ++j) {
                decay *= av[j];
                h[j] *= decay;
                dv[j] *= decay;
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                g.s[i][0] *= decay;
#pragma unroll
                for (int j = 0; j < GT; ++j) g.s[i][0] = fmaf(-kr[j][i], dv[j], g.s[i][0]);
            }
#pragma unroll
            for (int j = 0; j < GT; ++j) {
                float qr[R];
                get_rows<V>(qr, qs + (t + j) * D, rl);
#pragma unroll
                for (int i = 0; i < R; ++i) g.s[i][0] = fmaf(qr[i], h[j], g.s[i][0]);
            }
        }
    }
    g.store(a.dS0 + sbase, rl);
}

template <typename T, int D, int NC>
__global__ void __launch_bounds__(NC * RL) back_few_kernel(const Args a)
{
    extern __shared__ __align__(16) uint8_t shm[];
    __shared__ __align__(16) float al[TB], be[TB], gram[TB / GT][GT][GT];
    const int half = gridDim.x / 2;
    if ((int)blockIdx.x < half) reverse_few<T, D, NC>(a, blockIdx.x, shm, al, be, gram);
    else states_few<T, D, NC>(a, blockIdx.x - half, shm, al, be);
}

// The token gradients of one chunk of one head, from the S entering it and
// the adjoint of the S leaving it: rows of S and of G are independent here, so
// a thread holds 4 rows and every eighth float4 of columns.  Forward over the
// tokens for dq and alpha S dv, backward for G vtilde.
template <typename T, int D>
__global__ void __launch_bounds__(D * 2, D == 64 ? 4 : 2) token_grads_kernel(const Args a)
{
    constexpr int NTH = D * 2, V = D / (4 * RL), NW = NTH / 32, TB = kGradTokens;
    extern __shared__ __align__(16) uint8_t shm[];
    float (*dks)[D] = reinterpret_cast<float (*)[D]>(shm);       // [64] alpha S dv
    const Buffers<float, TB, D> fbuf{reinterpret_cast<float*>(shm + kChunk * D * 4)};  // dv
    const Buffers<T, TB, 4 * D> buf{reinterpret_cast<T*>(shm + (kChunk + 2 * TB) * D * 4)};  // do, vtilde, k, q
    __shared__ float al[TB], be[TB], dd[TB];
    __shared__ float bb[kChunk][NW];  // a warp's share of dbeta
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
#pragma unroll 2
        for (int t = 0; t < m; ++t) {
            float p[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};  // S do, S dv of the 4 rows
            const float alpha = al[t], b = be[t];
            const float4 k4 = get4(ks + t * D + row4);
            const float bk[4] = {b * k4.x, b * k4.y, b * k4.z, b * k4.w};
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = i * (4 * RL) + rl * 4;
                const float4 o4 = get4(c0 + t * D + c), d4 = get4(c1 + t * D + c), v4 = get4(c2 + t * D + c);
                const float vv[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float4 s4 = make_float4(s[r][4 * i], s[r][4 * i + 1], s[r][4 * i + 2], s[r][4 * i + 3]);
                    p[r] = dot4(s4, o4, p[r]);
                    p[4 + r] = dot4(s4, d4, p[4 + r]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[r][4 * i + e] = fmaf(alpha, s[r][4 * i + e], bk[r] * vv[e]);
                }
            }
            // lane r: dq of row r; lane 4 + r: alpha S dv of row r
            const float x = alpha * lanes_sum8(p, rl);
            const int row = row4 + rl % 4;
            const float kv = ld_elem(ks + t * D + row);
            const size_t tok = (size_t)(cr.row0 + t0 + t);
            if (rl < 4) {
                const float y = a.scale * fmaf(b * kv, dd[t], x);
                if (a.dqp) a.dqp[(tok * a.H + h) * D + row] = y;
                else st_elem(static_cast<T*>(a.dq) + (tok * a.Hk + hk) * D + row, y);
            } else {
                dks[t0 + t][row] = x;
            }
        }
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
#pragma unroll 2
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
            const float x = lanes_sum4(p, rl);
            const int row = row4 + rl % 4;
            const size_t tok = (size_t)(cr.row0 + t0 + t);
            float share = 0.f;
            if (rl < 4) {  // G vtilde of row rl
                const float z = fmaf(a.scale * ld_elem(qs + t * D + row), dd[t], x);
                share = ld_elem(ks + t * D + row) * z;
                const float y = fmaf(b, z, -dks[t0 + t][row]);
                if (a.dkp) a.dkp[(tok * a.H + h) * D + row] = y;
                else st_elem(static_cast<T*>(a.dk) + (tok * a.Hk + hk) * D + row, y);
            }
            share = warp_sum(share);
            if (lane == 0) bb[t0 + t][warp] = share;
        }
    }
    __syncthreads();
    for (int t = tid; t < cr.valid; t += NTH) {
        float b = 0.f;
        for (int w = 0; w < NW; ++w) b += bb[t][w];
        a.dbeta[(size_t)(cr.row0 + t) * a.H + h] = b;
    }
}

// dalpha_log of one chunk of one head: the sum of everything whose decay spans the token.
// With S entering and G leaving the chunk and L_{r,i} the decay from token i to token r,
//     Z_{r,i} = L_{r,i} beta_i (scale (do_r.vtilde_i) (q_r.k_i) - (dv_r.vtilde_i) (k_r.k_i)),  i < r,
//     e_r = L_{r,0} (scale q_r^T S do_r - k_r^T S dv_r),   f_i = L_{end,i} beta_i k_i^T G vtilde_i,
//     dalpha_log_t = L_{end,0} <G, S> + sum_{r >= t} e_r + sum_{i < t} f_i + sum_{r >= t > i} Z_{r,i}.
// (The recurrence dalpha_log_t = dalpha_log_{t+1} + q.dq - beta dbeta - ... needs no pairs, but
// adds and later takes off what each token does to itself, larger by 1 / alpha than what is
// left: at alpha = e^-8 it lost 1e-3 of the result.  A suffix sum of Z's row sums less its column
// sums does the same with the pairs behind t: one token of e^-8 among slow ones lost 1e-3.)
// Four threads a token; decays are running products, sums have a fixed order.  Bound by
// latency: 264 chunks of d 64 take 52 us.
template <typename T, int D>
__global__ void __launch_bounds__(256) dalpha_kernel(const Args a)
{
    constexpr int LD = D + 4, P = D / 4;  // P: a thread's columns
    extern __shared__ __align__(16) uint8_t shm[];
    float* ks = reinterpret_cast<float*>(shm);  // [64][LD] each
    float* qs = ks + kChunk * LD;
    float* vs = qs + kChunk * LD;
    float* os = vs + kChunk * LD;
    float* ds = os + kChunk * LD;
    float (*z)[kChunk + 1] = reinterpret_cast<float (*)[kChunk + 1]>(ds + kChunk * LD);
    __shared__ float al[kChunk], be[kChunk], e_[kChunk], f_[kChunk], rc[kChunk], gsum[8];
    const long long n = blockIdx.x / a.H;
    const int h = blockIdx.x % a.H, hk = h / (a.H / a.Hk);
    const ChunkRows cr = chunk_rows(a, n);
    if (cr.valid <= 0) return;
    const int tid = threadIdx.x, r = tid / 4, part = tid % 4;
    for (int x = tid; x < kChunk * (D / 4); x += 256) {
        const int t = x / (D / 4), c = x % (D / 4) * 4;
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        const bool in = t < cr.valid;
        const size_t kt = ((size_t)(cr.row0 + (in ? t : 0)) * a.Hk + hk) * D + c;
        const size_t vt = ((size_t)(cr.row0 + (in ? t : 0)) * a.H + h) * D + c;
        *reinterpret_cast<float4*>(ks + t * LD + c) = in ? get4(static_cast<const T*>(a.k) + kt) : zero;
        *reinterpret_cast<float4*>(qs + t * LD + c) = in ? get4(static_cast<const T*>(a.q) + kt) : zero;
        *reinterpret_cast<float4*>(vs + t * LD + c) = in ? get4(static_cast<const T*>(a.vt) + vt) : zero;
        *reinterpret_cast<float4*>(os + t * LD + c) = in ? get4(static_cast<const T*>(a.d_o) + vt) : zero;
        *reinterpret_cast<float4*>(ds + t * LD + c) = in ? get4(a.dvf + vt) : zero;
    }
    if (tid < kChunk) {
        const bool in = tid < cr.valid;
        const size_t at = (size_t)(cr.row0 + (in ? tid : 0)) * a.H + h;
        al[tid] = in ? expf(a.alpha_log[at]) : 1.f;
        be[tid] = in ? a.beta[at] : 0.f;
    }
    __syncthreads();
    auto sum4 = [](float x) {
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        return x + __shfl_xor_sync(0xffffffffu, x, 2);
    };
    {
        // S and G against this thread's token
        const float* S = a.SS + ((size_t)n * a.H + h) * D * D;
        const float* G = a.GG + ((size_t)n * a.H + h) * D * D;
        float o[P], d[P], v[P], es = 0.f, fs = 0.f;
#pragma unroll
        for (int c = 0; c < P; ++c) {
            const int y = 4 * part + c % 4 + c / 4 * 16;
            o[c] = a.scale * os[r * LD + y];
            d[c] = ds[r * LD + y];
            v[c] = vs[r * LD + y];
        }
        // 16 rows of both at a time through shared memory (where Z goes later), the next ones
        // on their way
        constexpr int TR = 16, NL = 2 * TR * D / 4 / 256;
        float* st = &z[0][0];
        static_assert(2 * TR * D <= kChunk * (kChunk + 1), "tile");
        float4 nx[NL];
        auto ahead = [&](int x0) {
#pragma unroll
            for (int l = 0; l < NL; ++l) {
                const int e = tid + 256 * l, of = e % (TR * D / 4) * 4;
                nx[l] = get4((e < TR * D / 4 ? S : G) + (size_t)x0 * D + of);
            }
        };
        ahead(0);
        float gs = 0.f;
        for (int x0 = 0; x0 < D; x0 += TR) {
            __syncthreads();
#pragma unroll
            for (int l = 0; l < NL; ++l) *reinterpret_cast<float4*>(st + 4 * (tid + 256 * l)) = nx[l];
            __syncthreads();
            if (x0 + TR < D) ahead(x0 + TR);
            for (int e = tid; e < TR * D / 4; e += 256) gs = dot4(get4(st + 4 * e), get4(st + TR * D + 4 * e), gs);
#pragma unroll 2
            for (int x = x0; x < x0 + TR; ++x) {
                float so = 0.f, sd = 0.f, gv = 0.f;
#pragma unroll
                for (int c = 0; c < P; c += 4) {
                    const float4 s4 = get4(st + (x - x0) * D + 4 * part + c * 4);
                    const float4 g4 = get4(st + TR * D + (x - x0) * D + 4 * part + c * 4);
                    so = dot4(s4, make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]), so);
                    sd = dot4(s4, make_float4(d[c], d[c + 1], d[c + 2], d[c + 3]), sd);
                    gv = dot4(g4, make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]), gv);
                }
                es += qs[r * LD + x] * so - ks[r * LD + x] * sd;
                fs = fmaf(ks[r * LD + x], gv, fs);
            }
        }
        es = sum4(es);
        fs = sum4(fs);
        float before = 1.f, after = 1.f;
        for (int t = 0; t < kChunk; ++t) {
            if (t <= r) before *= al[t];
            else after *= al[t];
        }
        if (part == 0) {
            e_[r] = before * es;
            f_[r] = after * be[r] * fs;
        }
        gs = warp_sum(gs);
        if (tid % 32 == 0) gsum[tid / 32] = before * after * gs;
    }
    __syncthreads();
    // pairs: this thread's token is i, r walks behind it; columns 4 part + 16 c of the rows
    {
        const int i = r;
        float L = 1.f;
        float4 vi[P / 4], ki[P / 4];
#pragma unroll
        for (int c = 0; c < P / 4; ++c) {
            vi[c] = get4(vs + i * LD + 4 * part + 16 * c);
            ki[c] = get4(ks + i * LD + 4 * part + 16 * c);
        }
        const int first = tid / 32 * 8 + 1;  // the warp's first token but one
        for (int t = part; t < first; t += 4) z[t][i] = 0.f;
#pragma unroll 2
        for (int t = first; t < kChunk; ++t) {
            float ov = 0.f, dv = 0.f, qk = 0.f, kk = 0.f;
#pragma unroll
            for (int c = 0; c < P / 4; ++c) {
                const int at = t * LD + 4 * part + 16 * c;
                ov = dot4(get4(os + at), vi[c], ov);
                dv = dot4(get4(ds + at), vi[c], dv);
                qk = dot4(get4(qs + at), ki[c], qk);
                kk = dot4(get4(ks + at), ki[c], kk);
            }
            if (t > i) L *= al[t];
            ov = sum4(ov); dv = sum4(dv); qk = sum4(qk); kk = sum4(kk);
            if (part == 0) z[t][i] = t > i ? L * be[i] * (a.scale * ov * qk - dv * kk) : 0.f;
        }
    }
    __syncthreads();
    {   // Z summed along each row inside its blocks of 16 columns, in place
        float* zr = &z[r][16 * part];
        float x = 0.f;
#pragma unroll
        for (int c = 0; c < 16; ++c) zr[c] = x += zr[c];
    }
    __syncthreads();
    {   // the pairs r2 >= r > i that span this thread's token r, and no others: four threads share the rows
        const int b = r / 16, in = r % 16;
        float x = 0.f;
        for (int t = r + part; t < kChunk; t += 4) {
            float y = in ? z[t][r - 1] : 0.f;
            for (int c = 0; c < b; ++c) y += z[t][16 * c + 15];
            x += y;
        }
        x = sum4(x);
        if (part == 0) rc[r] = x;
    }
    __syncthreads();
    if (tid < cr.valid) {
        float y = 0.f;
        for (int w = 0; w < 8; ++w) y += gsum[w];
        for (int t = 0; t < tid; ++t) y += f_[t];
        float x = rc[tid];
        for (int t = kChunk - 1; t >= tid; --t) x += e_[t];
        // nothing enters a sequence's first token from no state: its decay has no effect
        a.dalpha_log[(size_t)(cr.row0 + tid) * a.H + h] = tid == 0 && cr.first && !a.S0 ? 0.f : x + y;
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

// Few chains, as long as CTAs of 32 columns are at most two per SM: one column a thread
// and four tokens a reduction, so that a token costs a warp few instructions and little
// waiting.  At d 64 a token takes 0.17 us in the forward pass and 0.15 in the reverse
// chain, the states beside it (0.20, 0.23 and 0.09 for the states with a reduction per
// token and 32 columns a CTA); bound by a warp's own latency, 3.6 cycles an instruction
// with one warp per scheduler.  More chains: the whole head a CTA and four columns a
// thread, which reads each staged k and q once for four columns.  At the border, 256
// tokens forward: 74 chains of d 128 take 183 us (whole heads 218), 148 of d 64 92 us (86;
// in bf16 82 and 94).
template <typename T, int D>
cudaError_t fwd_typed(const Args& a, cudaStream_t s)
{
    const long long n = chains(a);
    ProfScope ps(kGdrFwdSimt, s);
    if (n * (D / 32) <= 2LL * sm_count())
        return run(fwd_few_kernel<T, D, kFew>, n * (D / kFew), kFew * RL, 2 * TB * (2 * D + kFew) * sizeof(T), s, a);
    return run(fwd_kernel<T, D>, n, 2 * D, 2 * TB * 3 * D * sizeof(T), s, a);
}

template <typename T, int D>
cudaError_t bwd_typed(const Args& a, cudaStream_t s)
{
    const long long n = chains(a);
    cudaError_t e;
    if (n * (D / 32) <= 2LL * sm_count()) {
        ProfScope ps(kGdrBwdChain, s);
        e = run(back_few_kernel<T, D, kFew>, 2 * n * (D / kFew), kFew * RL, 2 * TB * (2 * D + kFew) * sizeof(T), s, a);
        if (e != cudaSuccess) return e;
    } else {
        {
            ProfScope ps(kGdrBwdStates, s);
            e = run(states_kernel<T, D>, n, 2 * D, 2 * TB * 2 * D * sizeof(T), s, a);
            if (e != cudaSuccess) return e;
        }
        ProfScope ps(kGdrBwdChain, s);
        e = run(reverse_kernel<T, D>, n, 2 * D, 2 * TB * 3 * D * sizeof(T), s, a);
        if (e != cudaSuccess) return e;
    }
    const long long blocks = chunks(a) * a.H;
    if (blocks == 0) return cudaSuccess;
    ProfScope ps(kGdrBwdGrads, s);
    e = run(token_grads_kernel<T, D>, blocks, 2 * D,
            (kChunk + 2 * kGradTokens) * D * sizeof(float) + 2 * kGradTokens * 4 * D * sizeof(T), s, a);
    if (e != cudaSuccess) return e;
    return run(dalpha_kernel<T, D>, blocks, 256,
               (5 * kChunk * (D + 4) + kChunk * (kChunk + 1)) * sizeof(float), s, a);
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
