// Group norm with an activation over channels-last rows, forward and backward
// (include/mdn.h, mdn_group_norm_fwd / _bwd).  x is [N, L, C]; group g of row
// block n has the statistics of its L x C/G values:
//
//     xhat = (x - mean) rstd,  n = xhat w + b,  y = act(n)  or  n act(gate)
//
// and, with dn the cotangent of n, dh = dn w, m1 = avg(dh), m2 = avg(dh xhat)
// over the group:
//
//     dx = rstd (dh - m1 - xhat m2),  dw = sum dn xhat,  db = sum dn.
//
// Bound by HBM (a few dozen operations per element).  Two forms:
//  - tokens (L = 1, the mixer's output head by head): a group is one
//    contiguous run, held in the registers of 1..32 lanes, so every tensor is
//    read and written once;
//  - rows (any L): the values of a group lie in L separate runs, and a block
//    of rows is read by whole rows, each thread keeping its channels; partial
//    statistics per block go through the workspace, then a second pass reads
//    the rows again (from L2 while a call's tensors fit there).
// The tokens form takes the variance in fp32 about the mean, from registers.  The
// rows form sums a block's values and their squares in fp64 (an fp32 sum of squares
// about any one value loses the variance when that value lies far from the rest),
// keeps a block's (mean, sum of squared distances) in fp32 and joins those about
// the group's mean.  dw and db are summed per thread, per block and then over
// blocks in a fixed order, so results do not depend on timing.
#include <algorithm>
#include <type_traits>

#include "mdn_internal.cuh"
#include "sm100.cuh"

namespace mdn {
namespace gn {

struct Args {
    const void* x;
    const void* gate;   // or null
    const float* weight;  // both or neither
    const float* bias;
    int N, L, C, G;
    float eps;
    int act;
    void* y;
    float* mean;  // [N, G]
    float* rstd;
    // backward
    const void* dy;
    void* dx;
    void* dgate;
    float* dweight;
    float* dbias;
    // workspace
    float* part;   // rows form: [N, blocks, G, 2] (mean, M2) or (sum dh, sum dh xhat)
    float* wpart;  // backward: [partial rows, 2, C]
    int blocks;    // row blocks per n (rows form) / grid.x (tokens form)
    int prows;     // partial rows of wpart
};

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // values of a thread in flight at once (rows form)

// 1 / (1 + exp(-z)) by the hardware's approximate exponential and reciprocal (a few
// 1e-7 relative near 0, |z| 1e-7 in the tails, where the value is small; results below
// 2^-126 become 0): with the rounded functions the tokens form is bound by issue.
__device__ __forceinline__ float sigmoid(float z)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
template <int ACT>
__device__ __forceinline__ float act_of(float z)
{
    return ACT == MDN_ACT_SILU ? z * sigmoid(z) : z;
}
// act(z) and its derivative
template <int ACT>
__device__ __forceinline__ void act_grad(float z, float& f, float& df)
{
    f = z;
    df = 1.f;
    if (ACT == MDN_ACT_SILU) {
        const float sg = sigmoid(z);
        f = z * sg;
        df = sg * (1.f + z * (1.f - sg));
    }
}

// VEC consecutive elements as fp32 (one 16-byte access when VEC > 1).
template <typename T, int VEC>
__device__ __forceinline__ void ldv(const T* p, float* x)
{
    if constexpr (VEC == 1) {
        x[0] = ld_elem(p);
    } else if constexpr (sizeof(T) == 4) {
        const float4 w = *reinterpret_cast<const float4*>(p);
        x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&u[e]);
            x[2 * e] = __low2float(v);
            x[2 * e + 1] = __high2float(v);
        }
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void stv(T* p, const float* x)
{
    if constexpr (VEC == 1) {
        st_elem(p, x[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            u[e] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// VEC elements as loaded, to be widened later: what a prefetch keeps.
template <typename T, int VEC> struct RawOf { using type = uint4; };
template <typename T> struct RawOf<T, 1> { using type = T; };
template <typename T, int VEC>
__device__ __forceinline__ void ld_raw(const T* p, typename RawOf<T, VEC>::type& r)
{
    r = *reinterpret_cast<const typename RawOf<T, VEC>::type*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void widen(const typename RawOf<T, VEC>::type& r, float* x)
{
    ldv<T, VEC>(reinterpret_cast<const T*>(&r), x);
}

// Sum over `lanes` (a power of two) neighbouring lanes, in each of them.
__device__ __forceinline__ float sum_lanes(float x, int lanes)
{
    for (int off = 1; off < lanes; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// ---------------------------------------------------------------- tokens form (L = 1)
// One lane group per (group slot, token slot); a lane keeps its channels, and so
// its weights, over all tokens it takes.  grid.y tiles the groups, grid.x the
// tokens.  TOK tokens at a time, so that their loads are in flight together.
template <typename T, int VEC, int NV, int TOK, int ACT, bool GATE>
__global__ void __launch_bounds__(kThreads, NV * VEC <= 8 ? 4 : 2) tokens_fwd_kernel(const Args a, int lanes, int gslots)
{
    const int Cg = a.C / a.G, units = Cg / VEC;
    const int lane = threadIdx.x % lanes, slot = threadIdx.x / lanes;
    const int per = kThreads / lanes / gslots;
    const int g = blockIdx.y * gslots + slot % gslots, ts = slot / gslots;
    const bool glive = g < a.G;
    float w[NV * VEC], b[NV * VEC];
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) {
        const int c = ((i / VEC) * lanes + lane) * VEC + i % VEC;
        const bool in = a.weight && glive && c < Cg;
        w[i] = in ? a.weight[(size_t)g * Cg + c] : 1.f;
        b[i] = in ? a.bias[(size_t)g * Cg + c] : 0.f;
    }
    const T* __restrict__ xin = static_cast<const T*>(a.x);
    const T* __restrict__ gin = static_cast<const T*>(a.gate);
    T* __restrict__ yout = static_cast<T*>(a.y);
    const int step = gridDim.x * per;
    const float inv = 1.f / Cg;
    using Raw = typename RawOf<T, VEC>::type;
    Raw xr[TOK][NV], zr[TOK][NV];
    auto fetch = [&](int n0) {
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            const int n = n0 + t * step + blockIdx.x * per + ts;
            const size_t at = ((size_t)n * a.G + g) * Cg;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int u = i * lanes + lane;
                if (glive && n < a.N && u < units) {
                    ld_raw<T, VEC>(xin + at + u * VEC, xr[t][i]);
                    if (GATE) ld_raw<T, VEC>(gin + at + u * VEC, zr[t][i]);
                }
            }
        }
    };
    fetch(0);
    for (int n0 = 0; n0 < a.N; n0 += step * TOK) {  // uniform trip count: shuffles below
        float v[TOK][NV * VEC], z[TOK][NV * VEC];
        size_t base[TOK];
        bool live[TOK];
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            const int n = n0 + t * step + blockIdx.x * per + ts;
            live[t] = glive && n < a.N;
            base[t] = ((size_t)n * a.G + g) * Cg;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (live[t] && i * lanes + lane < units) {
                    widen<T, VEC>(xr[t][i], v[t] + i * VEC);
                    if (GATE) widen<T, VEC>(zr[t][i], z[t] + i * VEC);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[t][i * VEC + e] = 0.f;
                }
            }
        }
        if (n0 + step * TOK < a.N) fetch(n0 + step * TOK);  // the next tokens, under this work
        float s[TOK], q[TOK];
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            s[t] = 0.f;
#pragma unroll
            for (int i = 0; i < NV * VEC; ++i) s[t] += v[t][i];
        }
        for (int off = 1; off < lanes; off <<= 1)
#pragma unroll
            for (int t = 0; t < TOK; ++t) s[t] += __shfl_xor_sync(0xffffffffu, s[t], off);
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            s[t] *= inv;
            q[t] = 0.f;
#pragma unroll
            for (int i = 0; i < NV * VEC; ++i) {
                const float d = v[t][i] - s[t];
                if ((i / VEC) * lanes + lane < units) q[t] = fmaf(d, d, q[t]);
            }
        }
        for (int off = 1; off < lanes; off <<= 1)
#pragma unroll
            for (int t = 0; t < TOK; ++t) q[t] += __shfl_xor_sync(0xffffffffu, q[t], off);
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            if (!live[t]) continue;
            const float mean = s[t], rstd = rsqrtf(q[t] * inv + a.eps);
            if (lane == 0) {
                const size_t item = (size_t)(n0 + t * step + blockIdx.x * per + ts) * a.G + g;
                a.mean[item] = mean;
                a.rstd[item] = rstd;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int u = i * lanes + lane;
                if (u >= units) continue;
                float y[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int j = i * VEC + e;
                    const float nn = fmaf((v[t][j] - mean) * rstd, w[j], b[j]);
                    y[e] = GATE ? nn * act_of<ACT>(z[t][j]) : act_of<ACT>(nn);
                }
                stv<T, VEC>(yout + base[t] + u * VEC, y);
            }
        }
    }
}

// The same mapping backward: dw and db add up in registers over a lane's tokens,
// then over the block's token slots in shared memory.
template <typename T, int VEC, int NV, int ACT, bool GATE>
__global__ void __launch_bounds__(kThreads) tokens_bwd_kernel(const Args a, int lanes, int gslots)
{
    sm100::pdl_launch_dependents();
    const int Cg = a.C / a.G, units = Cg / VEC;
    const int lane = threadIdx.x % lanes, slot = threadIdx.x / lanes;
    const int per = kThreads / lanes / gslots;  // token slots of the block
    const int g = blockIdx.y * gslots + slot % gslots, ts = slot / gslots;
    const bool glive = g < a.G;
    const int prow = blockIdx.x * per + ts;
    float w[NV * VEC], b[NV * VEC], dw[NV * VEC], db[NV * VEC];
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) {
        dw[i] = db[i] = 0.f;
        const int c = ((i / VEC) * lanes + lane) * VEC + i % VEC;
        w[i] = 1.f;
        b[i] = 0.f;
        if (a.weight && glive && c < Cg) {
            w[i] = a.weight[(size_t)g * Cg + c];
            b[i] = a.bias[(size_t)g * Cg + c];
        }
    }
    const T* __restrict__ xin = static_cast<const T*>(a.x);
    const T* __restrict__ dyin = static_cast<const T*>(a.dy);
    const T* __restrict__ gin = static_cast<const T*>(a.gate);
    const int step = gridDim.x * per;
    const float inv = 1.f / Cg;
    using Raw = typename RawOf<T, VEC>::type;
    Raw xr[NV], dr[NV], zr[NV];
    float mr[2] = {0.f, 0.f};
    auto fetch = [&](int n) {
        if (!(glive && n < a.N)) return;
        const size_t at = ((size_t)n * a.G + g) * Cg;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = i * lanes + lane;
            if (u < units) {
                ld_raw<T, VEC>(xin + at + u * VEC, xr[i]);
                ld_raw<T, VEC>(dyin + at + u * VEC, dr[i]);
                if (GATE) ld_raw<T, VEC>(gin + at + u * VEC, zr[i]);
            }
        }
        mr[0] = a.mean[(size_t)n * a.G + g];
        mr[1] = a.rstd[(size_t)n * a.G + g];
    };
    fetch(prow);
    for (int n0 = 0; n0 < a.N; n0 += step) {  // uniform trip count: shuffles below
        const int n = n0 + prow;
        const bool live = glive && n < a.N;
        const size_t base = ((size_t)n * a.G + g) * Cg;
        const float mean = mr[0], rstd = mr[1];
        float xh[NV * VEC], dh[NV * VEC], z[NV * VEC];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && i * lanes + lane < units) {
                widen<T, VEC>(xr[i], xh + i * VEC);
                widen<T, VEC>(dr[i], dh + i * VEC);
                if (GATE) widen<T, VEC>(zr[i], z + i * VEC);
            }
        if (n0 + step < a.N) fetch(n + step);  // the next token, under this one's work
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = i * lanes + lane;
            if (!(live && u < units)) continue;
            float dz[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int j = i * VEC + e;
                const float h = (xh[j] - mean) * rstd, nn = fmaf(h, w[j], b[j]);
                float f, df, dn;
                act_grad<ACT>(GATE ? z[j] : nn, f, df);
                if (GATE) {
                    dn = dh[j] * f;
                    dz[e] = dh[j] * nn * df;
                } else {
                    dn = dh[j] * df;
                }
                dw[j] = fmaf(dn, h, dw[j]);
                db[j] += dn;
                xh[j] = h;
                dh[j] = dn * w[j];
                s1 += dh[j];
                s2 = fmaf(dh[j], h, s2);
            }
            if (GATE) stv<T, VEC>(static_cast<T*>(a.dgate) + base + u * VEC, dz);
        }
        const float m1 = sum_lanes(s1, lanes) * inv, m2 = sum_lanes(s2, lanes) * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = i * lanes + lane;
            if (!(live && u < units)) continue;
            float dx[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                dx[e] = rstd * (dh[i * VEC + e] - m1 - xh[i * VEC + e] * m2);
            stv<T, VEC>(static_cast<T*>(a.dx) + base + u * VEC, dx);
        }
    }
    if (!a.dweight) return;
    extern __shared__ float sh[];  // [2 NV VEC][kThreads]
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) {
        sh[2 * i * kThreads + threadIdx.x] = dw[i];
        sh[(2 * i + 1) * kThreads + threadIdx.x] = db[i];
    }
    __syncthreads();
    if (ts != 0 || !glive) return;
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) {
        const int c = ((i / VEC) * lanes + lane) * VEC + i % VEC;
        if (c >= Cg) continue;
        float x = 0.f, y = 0.f;
        for (int t = 0; t < per; ++t) {  // token slots in order
            x += sh[2 * i * kThreads + threadIdx.x + t * gslots * lanes];
            y += sh[(2 * i + 1) * kThreads + threadIdx.x + t * gslots * lanes];
        }
        a.wpart[((size_t)blockIdx.x * 2) * a.C + (size_t)g * Cg + c] = x;
        a.wpart[((size_t)blockIdx.x * 2 + 1) * a.C + (size_t)g * Cg + c] = y;
    }
}

// The tokens form for groups of exactly LANES vectors (a power of two: head sizes).
// The same mapping with nothing left to test per element: 32768 x 2048 gated bf16 (403 MB)
// take 71 us forward instead of 94, 5.7 TB/s; ungated 62 us (issue- and special-function-
// bound: an exponential and a reciprocal per value).  The grid is what runs at once.
// Backward keeps two tokens in flight per thread, as its registers admit two blocks per
// SM only: 8192 x 1024 gated bf16 26.5 us instead of 28.5 with one.
template <typename T, int LANES, int ACT, bool GATE, bool BWD>
__global__ void __launch_bounds__(kThreads, BWD ? 2 : 4) tokens_exact_kernel(const Args a, int gslots)
{
    constexpr int V = 16 / (int)sizeof(T), Cg = LANES * V;
    constexpr float inv = 1.f / Cg;
    if (BWD) sm100::pdl_launch_dependents();
    constexpr int AHEAD = BWD ? 2 : 1;  // tokens in flight per thread
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    const int per = kThreads / LANES / gslots;
    const int g = blockIdx.y * gslots + slot % gslots, ts = slot / gslots;
    const bool glive = g < a.G;
    float w[V], b[V], dw[V], db[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const bool in = a.weight && glive;
        w[e] = in ? a.weight[(size_t)g * Cg + lane * V + e] : 1.f;
        b[e] = in ? a.bias[(size_t)g * Cg + lane * V + e] : 0.f;
        dw[e] = db[e] = 0.f;
    }
    const int step = gridDim.x * per;
    long long n = (long long)blockIdx.x * per + ts;
    const size_t hop = (size_t)step * a.G;
    size_t item = (size_t)n * a.G + g;
    struct Raw {
        uint4 x, z, d;
        float mean, rstd;
    } raw[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) raw[u] = Raw{};
    auto fetch = [&](Raw& f, long long n_, size_t it) {
        if (!(glive && n_ < a.N)) return;
        const size_t at = it * Cg + lane * V;
        f.x = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + at);
        if (GATE) f.z = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.gate) + at);
        if (BWD) {
            f.d = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.dy) + at);
            f.mean = a.mean[it];
            f.rstd = a.rstd[it];
        }
    };
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) fetch(raw[u], n + (long long)u * step, item + u * hop);
    auto token = [&](Raw& f) {
        const bool live = glive && n < a.N;
        float v[V], z[V], d[V];
        widen<T, V>(f.x, v);
        if (GATE) widen<T, V>(f.z, z);
        if (BWD) widen<T, V>(f.d, d);
        float mean = f.mean, rstd = f.rstd;
        fetch(f, n + (long long)AHEAD * step, item + AHEAD * hop);
        const size_t at = item * Cg + lane * V;
        if (!BWD) {
            float s = 0.f, q = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) s += v[e];
#pragma unroll
            for (int off = 1; off < LANES; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            mean = s * inv;
#pragma unroll
            for (int e = 0; e < V; ++e) q = fmaf(v[e] - mean, v[e] - mean, q);
#pragma unroll
            for (int off = 1; off < LANES; off <<= 1) q += __shfl_xor_sync(0xffffffffu, q, off);
            rstd = rsqrtf(q * inv + a.eps);
            if (!live) return;
            if (lane == 0) {
                a.mean[item] = mean;
                a.rstd[item] = rstd;
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float nn = fmaf((v[e] - mean) * rstd, w[e], b[e]);
                v[e] = GATE ? nn * act_of<ACT>(z[e]) : act_of<ACT>(nn);
            }
            stv<T, V>(static_cast<T*>(a.y) + at, v);
        } else {
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float h = (v[e] - mean) * rstd, nn = fmaf(h, w[e], b[e]);
                float f, df, dn;
                act_grad<ACT>(GATE ? z[e] : nn, f, df);
                dn = d[e] * (GATE ? f : df);
                if (GATE) z[e] = d[e] * nn * df;
                if (!live) dn = 0.f;
                dw[e] = fmaf(dn, h, dw[e]);
                db[e] += dn;
                v[e] = h;
                d[e] = dn * w[e];
                s1 += d[e];
                s2 = fmaf(d[e], h, s2);
            }
#pragma unroll
            for (int off = 1; off < LANES; off <<= 1) {
                s1 += __shfl_xor_sync(0xffffffffu, s1, off);
                s2 += __shfl_xor_sync(0xffffffffu, s2, off);
            }
            if (!live) return;
            if (GATE) stv<T, V>(static_cast<T*>(a.dgate) + at, z);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = rstd * (d[e] - s1 * inv - v[e] * (s2 * inv));
            stv<T, V>(static_cast<T*>(a.dx) + at, v);
        }
    };
    for (long long n0 = 0; n0 < a.N;) {  // uniform: shuffles in token()
#pragma unroll
        for (int u = 0; u < AHEAD; ++u, n0 += step, n += step, item += hop) token(raw[u]);
    }
    if (!BWD || !a.dweight) return;
    extern __shared__ float sh[];  // [2 V][kThreads]
#pragma unroll
    for (int e = 0; e < V; ++e) {
        sh[2 * e * kThreads + threadIdx.x] = dw[e];
        sh[(2 * e + 1) * kThreads + threadIdx.x] = db[e];
    }
    __syncthreads();
    if (ts != 0 || !glive) return;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float x = 0.f, y = 0.f;
        for (int t = 0; t < per; ++t) {  // token slots in order
            x += sh[2 * e * kThreads + threadIdx.x + t * gslots * LANES];
            y += sh[(2 * e + 1) * kThreads + threadIdx.x + t * gslots * LANES];
        }
        a.wpart[((size_t)blockIdx.x * 2) * a.C + (size_t)g * Cg + lane * V + e] = x;
        a.wpart[((size_t)blockIdx.x * 2 + 1) * a.C + (size_t)g * Cg + lane * V + e] = y;
    }
}

// ---------------------------------------------------------------- rows form
// Block (blk, n) covers rows [l0, l1) of n; grid.z tiles the channels by
// kThreads.  A thread owns one channel; threads of a group join in shared
// memory, in channel order.
struct RowBlock {
    int l0, l1;
};
__device__ __forceinline__ RowBlock row_block(const Args& a)
{
    const int per = (a.L + a.blocks - 1) / a.blocks;
    RowBlock r;
    r.l0 = min(a.L, (int)blockIdx.x * per);
    r.l1 = min(a.L, r.l0 + per);
    return r;
}

// Partial statistics.  One warp per (n, group, row block): the lanes take the
// group's values of the block in turn.
template <typename T, bool BWD, int ACT, bool GATE>
__global__ void __launch_bounds__(kThreads) rows_part_kernel(const Args a)
{
    sm100::pdl_launch_dependents();
    const int Cg = a.C / a.G, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = blockIdx.z * (kThreads / 32) + warp, n = blockIdx.y;
    if (g >= a.G) return;
    const RowBlock rb = row_block(a);
    const int rows = rb.l1 - rb.l0;
    const T* x = static_cast<const T*>(a.x);
    const size_t base = ((size_t)n * a.L + rb.l0) * a.C + (size_t)g * Cg;
    const long long cnt = (long long)rows * Cg;
    // lane's first value and the step from value to value, as (row, channel)
    int r = lane / Cg, c = lane % Cg;
    const int sr = 32 / Cg, sc = 32 % Cg;
    float* out = a.part + (((size_t)n * a.blocks + blockIdx.x) * a.G + g) * 2;
    if constexpr (!BWD) {
        // Q - P mean keeps 53 - 2 log2(|mean| / spread) bits: 24 of them at a mean of 2^14 spreads
        double p = 0.0, q = 0.0;
        for (long long i = lane; i < cnt; i += 32 * kBatch) {
            float v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                v[u] = i + 32 * u < cnt ? ld_elem(x + base + (size_t)r * a.C + c) : 0.f;
                r += sr; c += sc;
                if (c >= Cg) { c -= Cg; ++r; }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const double w = v[u];
                p += w;
                q = fma(w, w, q);
            }
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            p += __shfl_xor_sync(0xffffffffu, p, off);
            q += __shfl_xor_sync(0xffffffffu, q, off);
        }
        if (lane == 0 && cnt > 0) {
            const double mean = p / (double)cnt, m2 = q - p * mean;
            out[0] = (float)mean;
            out[1] = (float)(m2 < 0.0 ? 0.0 : m2);  // keeps a NaN
        }
    } else {
        const T* dy = static_cast<const T*>(a.dy);
        const T* gate = static_cast<const T*>(a.gate);
        const float mean = a.mean[(size_t)n * a.G + g], rstd = a.rstd[(size_t)n * a.G + g];
        float p = 0.f, q = 0.f;
        for (long long i = lane; i < cnt; i += 32 * kBatch) {
            float xv[kBatch], dv[kBatch], zv[kBatch], wv[kBatch], bv[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const size_t at = base + (size_t)r * a.C + c;
                const bool in = i + 32 * u < cnt;
                xv[u] = in ? ld_elem(x + at) : mean;
                dv[u] = in ? ld_elem(dy + at) : 0.f;
                zv[u] = in && GATE ? ld_elem(gate + at) : 0.f;
                wv[u] = in && a.weight ? a.weight[(size_t)g * Cg + c] : 1.f;
                bv[u] = in && a.weight ? a.bias[(size_t)g * Cg + c] : 0.f;
                r += sr; c += sc;
                if (c >= Cg) { c -= Cg; ++r; }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const float h = (xv[u] - mean) * rstd;
                float f, df;
                act_grad<ACT>(GATE ? zv[u] : fmaf(h, wv[u], bv[u]), f, df);
                const float dh = i + 32 * u < cnt ? dv[u] * (GATE ? f : df) * wv[u] : 0.f;
                p += dh;
                q = fmaf(dh, h, q);
            }
        }
        p = sum_lanes(p, 32);
        q = sum_lanes(q, 32);
        if (lane == 0) {
            out[0] = p;
            out[1] = q;
        }
    }
}

// The (n, group) statistics of the block's groups, from all row blocks, in
// shared memory (a warp per group, its lanes over the row blocks); forward: mean
// and rstd, written out by the first row block.
template <bool BWD>
__device__ __forceinline__ void join_parts(const Args& a, int n, int g0, int g1, float2* st)
{
    const int Cg = a.C / a.G, per = (a.L + a.blocks - 1) / a.blocks, lane = threadIdx.x % 32;
    for (int g = g0 + (int)threadIdx.x / 32; g < g1; g += kThreads / 32) {
        const float2* p = reinterpret_cast<const float2*>(a.part) + (size_t)n * a.blocks * a.G + g;
        if constexpr (!BWD) {
            // sums about the first block's mean, then about the group's
            const float e0 = p[0].x, all = (float)a.L * Cg;
            auto count = [&](int b) { return (float)max(0, min(a.L, (b + 1) * per) - min(a.L, b * per)) * Cg; };
            float s = 0.f, m2 = 0.f;
            for (int b = lane; b < a.blocks; b += 32) {
                const float k = count(b);
                if (k > 0.f) s = fmaf(k, p[(size_t)b * a.G].x - e0, s);
            }
            const float mean = e0 + sum_lanes(s, 32) / all;
            for (int b = lane; b < a.blocks; b += 32) {
                const float2 v = p[(size_t)b * a.G];
                const float k = count(b), d = v.x - mean;
                if (k > 0.f) m2 += fmaf(k * d, d, v.y);
            }
            m2 = sum_lanes(m2, 32);
            const float rstd = rsqrtf(m2 / all + a.eps);
            if (lane == 0) {
                st[g - g0] = make_float2(mean, rstd);
                if (blockIdx.x == 0) {
                    a.mean[(size_t)n * a.G + g] = mean;
                    a.rstd[(size_t)n * a.G + g] = rstd;
                }
            }
        } else {
            float s = 0.f, q = 0.f;
            for (int b = lane; b < a.blocks; b += 32) {
                const float2 v = p[(size_t)b * a.G];
                s += v.x;
                q += v.y;
            }
            s = sum_lanes(s, 32);
            q = sum_lanes(q, 32);
            const float m = (float)a.L * Cg;
            if (lane == 0) st[g - g0] = make_float2(s / m, q / m);
        }
    }
    __syncthreads();
}

// The second pass.  Its rows do not depend on the first, so the first batch of them is
// in flight while the statistics are joined, and each further one while its forerunner
// is worked on.
template <typename T, int ACT, bool GATE>
__global__ void __launch_bounds__(kThreads) rows_fwd_kernel(const Args a)
{
    __shared__ float2 st[kThreads];  // a tile of kThreads channels touches at most as many groups
    const int Cg = a.C / a.G, n = blockIdx.y, c = blockIdx.z * kThreads + threadIdx.x;
    const int g0 = blockIdx.z * kThreads / Cg;
    const int g1 = (min(a.C, (int)(blockIdx.z + 1) * kThreads) - 1) / Cg + 1;
    const RowBlock rb = row_block(a);
    const int l1 = c < a.C ? rb.l1 : 0;
    const T* x = static_cast<const T*>(a.x);
    const T* gate = static_cast<const T*>(a.gate);
    size_t at = ((size_t)n * a.L + rb.l0) * a.C + c;
    float xn[kBatch], zn[kBatch];
    auto fetch = [&](int l, size_t from) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const bool in = l + u < l1;
            xn[u] = in ? ld_elem(x + from + (size_t)u * a.C) : 0.f;
            if (GATE) zn[u] = in ? ld_elem(gate + from + (size_t)u * a.C) : 0.f;
        }
    };
    fetch(rb.l0, at);
    const float w = a.weight && c < a.C ? a.weight[c] : 1.f, b = a.weight && c < a.C ? a.bias[c] : 0.f;
    sm100::pdl_wait();  // for the partial statistics
    join_parts<false>(a, n, g0, g1, st);
    if (c >= a.C) return;
    const float2 ms = st[c / Cg - g0];
    for (int l = rb.l0; l < l1; l += kBatch, at += (size_t)kBatch * a.C) {
        float xv[kBatch], zv[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            xv[u] = xn[u];
            if (GATE) zv[u] = zn[u];
        }
        fetch(l + kBatch, at + (size_t)kBatch * a.C);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (l + u >= l1) break;
            const float nn = fmaf((xv[u] - ms.x) * ms.y, w, b);
            st_elem(static_cast<T*>(a.y) + at + (size_t)u * a.C,
                    GATE ? nn * act_of<ACT>(zv[u]) : act_of<ACT>(nn));
        }
    }
}

template <typename T, int ACT, bool GATE>
__global__ void __launch_bounds__(kThreads) rows_bwd_kernel(const Args a)
{
    __shared__ float2 st[kThreads];
    const int Cg = a.C / a.G, n = blockIdx.y, c = blockIdx.z * kThreads + threadIdx.x;
    const int g0 = blockIdx.z * kThreads / Cg;
    const int g1 = (min(a.C, (int)(blockIdx.z + 1) * kThreads) - 1) / Cg + 1;
    const RowBlock rb = row_block(a);
    const int l1 = c < a.C ? rb.l1 : 0;
    const T* x = static_cast<const T*>(a.x);
    const T* dy = static_cast<const T*>(a.dy);
    const T* gate = static_cast<const T*>(a.gate);
    size_t at = ((size_t)n * a.L + rb.l0) * a.C + c;
    float xn[kBatch], dn_[kBatch], zn[kBatch];
    auto fetch = [&](int l, size_t from) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const bool in = l + u < l1;
            xn[u] = in ? ld_elem(x + from + (size_t)u * a.C) : 0.f;
            dn_[u] = in ? ld_elem(dy + from + (size_t)u * a.C) : 0.f;
            if (GATE) zn[u] = in ? ld_elem(gate + from + (size_t)u * a.C) : 0.f;
        }
    };
    sm100::pdl_launch_dependents();
    fetch(rb.l0, at);
    const int g = c / Cg;
    float w = 1.f, b = 0.f, mean = 0.f, rstd = 0.f;
    if (c < a.C) {
        if (a.weight) w = a.weight[c], b = a.bias[c];
        mean = a.mean[(size_t)n * a.G + g];
        rstd = a.rstd[(size_t)n * a.G + g];
    }
    sm100::pdl_wait();  // for the partial sums
    join_parts<true>(a, n, g0, g1, st);
    if (c >= a.C) return;
    const float2 m = st[g - g0];
    float dw = 0.f, db = 0.f;
    for (int l = rb.l0; l < l1; l += kBatch, at += (size_t)kBatch * a.C) {
        float xv[kBatch], dv[kBatch], zv[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            xv[u] = xn[u];
            dv[u] = dn_[u];
            if (GATE) zv[u] = zn[u];
        }
        fetch(l + kBatch, at + (size_t)kBatch * a.C);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (l + u >= l1) break;
            const size_t to = at + (size_t)u * a.C;
            const float h = (xv[u] - mean) * rstd, nn = fmaf(h, w, b);
            float f, df;
            act_grad<ACT>(GATE ? zv[u] : nn, f, df);
            const float dn = dv[u] * (GATE ? f : df);
            if (GATE) st_elem(static_cast<T*>(a.dgate) + to, dv[u] * nn * df);
            dw = fmaf(dn, h, dw);
            db += dn;
            st_elem(static_cast<T*>(a.dx) + to, rstd * (dn * w - m.x - h * m.y));
        }
    }
    if (a.dweight) {
        const size_t prow = (size_t)n * a.blocks + blockIdx.x;
        a.wpart[prow * 2 * a.C + c] = dw;
        a.wpart[(prow * 2 + 1) * a.C + c] = db;
    }
}

// dweight, dbias: the partial rows of a channel, 32 at a time, in a fixed order.
__global__ void __launch_bounds__(1024) wsum_kernel(const Args a)
{
    __shared__ float sh[32][33];
    const long long c = (long long)blockIdx.x * 32 + threadIdx.x % 32;  // of [2, C]
    const int r0 = threadIdx.x / 32;
    float s = 0.f;
    sm100::pdl_wait();  // for the partial rows
    if (c < 2LL * a.C)
        for (int r = r0; r < a.prows; r += 32 * 8) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = r + 32 * u < a.prows ? a.wpart[(size_t)(r + 32 * u) * 2 * a.C + c] : 0.f;
#pragma unroll
            for (int u = 0; u < 8; ++u) s += v[u];
        }
    sh[r0][threadIdx.x % 32] = s;
    __syncthreads();
    s = sh[threadIdx.x % 32][r0];
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const long long d = (long long)blockIdx.x * 32 + r0;
    if (threadIdx.x % 32 == 0 && d < 2LL * a.C) *(d < a.C ? a.dweight + d : a.dbias + (d - a.C)) = s;
}

// How a call runs: the tokens form's lanes and vectors, or the rows form.
struct Plan {
    bool tokens;
    bool vec;     // 16-byte vectors (the group's length and the pointers allow them)
    int lanes, nv;
    int gslots;   // tokens form: group slots of a block, tiles of groups
    int gtiles;
    int blocks;   // row blocks per n (rows form), token blocks (tokens form)
    int prows;    // partial rows of dw, db
    size_t part_bytes, bytes;
};

// vec is a property of the pointers, so the workspace is sized for both.
Plan plan_of(int N, int L, int C, int G, bool f32, bool vec, bool bwd)
{
    Plan p = {};
    const int Cg = C / G, V = f32 ? 4 : 8;
    p.vec = vec && Cg % V == 0;
    const int units = p.vec ? Cg / V : Cg;
    p.lanes = 1;
    while (p.lanes < 32 && p.lanes < units) p.lanes <<= 1;
    p.nv = (units + p.lanes - 1) / p.lanes;
    p.tokens = L == 1 && p.nv <= (p.vec ? 2 : 8);
    const int want = 148 * 4;  // blocks that keep every SM busy
    if (p.tokens) {
        p.nv = p.vec ? (p.nv <= 1 ? 1 : 2) : (p.nv <= 4 ? 4 : 8);
        const int slots = kThreads / p.lanes;
        p.gslots = 1;
        while (p.gslots < slots && p.gslots < G) p.gslots <<= 1;
        p.gtiles = (G + p.gslots - 1) / p.gslots;
        const int per = slots / p.gslots;
        const int most = (N + per - 1) / per;
        // as many blocks as run at once, several tokens each
        p.blocks = std::max(1, std::min(most, std::max(1, 148 * (bwd ? 2 : 4) / p.gtiles)));
        p.prows = p.blocks;
    } else {
        // rows per block at least 16: the second pass rereads the partials of every block
        const int ctiles = (C + kThreads - 1) / kThreads;
        const long long others = (long long)N * ctiles;
        p.blocks = (int)std::max(1LL, std::min<long long>((L + 15) / 16, (want + others - 1) / others));
        p.prows = N * p.blocks;
        p.part_bytes = ((size_t)N * p.blocks * G * 2 * sizeof(float) + 255) / 256 * 256;
    }
    p.bytes = p.part_bytes + (bwd ? (size_t)p.prows * 2 * C * sizeof(float) : 0);
    return p;
}

size_t workspace_bytes(int N, int L, int C, int G, bool f32, bool bwd)
{
    return std::max(plan_of(N, L, C, G, f32, true, bwd).bytes, plan_of(N, L, C, G, f32, false, bwd).bytes);
}

// The exact tokens form, if the groups are whole vectors of 4..32 lanes.
template <typename T, int ACT, bool GATE, bool BWD>
bool launch_exact(const Args& a, const Plan& p, cudaStream_t s)
{
    constexpr int V = 16 / (int)sizeof(T);
    if (!p.tokens || !p.vec || a.C / a.G != p.lanes * V || p.lanes < 4) return false;
    const dim3 grid(p.blocks, p.gtiles);
    const size_t shm = BWD && a.dweight ? (size_t)2 * V * kThreads * sizeof(float) : 0;
    if (p.lanes == 4) tokens_exact_kernel<T, 4, ACT, GATE, BWD><<<grid, kThreads, shm, s>>>(a, p.gslots);
    else if (p.lanes == 8) tokens_exact_kernel<T, 8, ACT, GATE, BWD><<<grid, kThreads, shm, s>>>(a, p.gslots);
    else if (p.lanes == 16) tokens_exact_kernel<T, 16, ACT, GATE, BWD><<<grid, kThreads, shm, s>>>(a, p.gslots);
    else tokens_exact_kernel<T, 32, ACT, GATE, BWD><<<grid, kThreads, shm, s>>>(a, p.gslots);
    return true;
}

template <typename T, int ACT, bool GATE>
cudaError_t fwd_typed(const Args& a, const Plan& p, cudaStream_t s)
{
    constexpr int V = 16 / (int)sizeof(T);
    ProfScope ps(kGroupNorm, s);
    if (launch_exact<T, ACT, GATE, false>(a, p, s)) return cudaGetLastError();
    if (p.tokens) {
        const dim3 grid(p.blocks, p.gtiles);
        if (p.vec && p.nv == 1) tokens_fwd_kernel<T, V, 1, 1, ACT, GATE><<<grid, kThreads, 0, s>>>(a, p.lanes, p.gslots);
        else if (p.vec) tokens_fwd_kernel<T, V, 2, 1, ACT, GATE><<<grid, kThreads, 0, s>>>(a, p.lanes, p.gslots);
        else if (p.nv == 4) tokens_fwd_kernel<T, 1, 4, 2, ACT, GATE><<<grid, kThreads, 0, s>>>(a, p.lanes, p.gslots);
        else tokens_fwd_kernel<T, 1, 8, 1, ACT, GATE><<<grid, kThreads, 0, s>>>(a, p.lanes, p.gslots);
        return cudaGetLastError();
    }
    const dim3 g1(p.blocks, a.N, (a.G + kThreads / 32 - 1) / (kThreads / 32));
    rows_part_kernel<T, false, ACT, GATE><<<g1, kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_dependent(rows_fwd_kernel<T, ACT, GATE>, dim3(p.blocks, a.N, (a.C + kThreads - 1) / kThreads),
                            kThreads, 0, s, a);
}

template <typename T, int ACT, bool GATE>
cudaError_t bwd_typed(const Args& a, const Plan& p, cudaStream_t s)
{
    constexpr int V = 16 / (int)sizeof(T);
    ProfScope ps(kGroupNormBwd, s);
    cudaError_t e;
    if (launch_exact<T, ACT, GATE, true>(a, p, s)) {
    } else if (p.tokens) {
        const dim3 grid(p.blocks, p.gtiles);
        const size_t shm = a.dweight ? (size_t)2 * p.nv * (p.vec ? V : 1) * kThreads * sizeof(float) : 0;
        if (p.vec && p.nv == 1) tokens_bwd_kernel<T, V, 1, ACT, GATE><<<grid, kThreads, shm, s>>>(a, p.lanes, p.gslots);
        else if (p.vec) tokens_bwd_kernel<T, V, 2, ACT, GATE><<<grid, kThreads, shm, s>>>(a, p.lanes, p.gslots);
        else if (p.nv == 4) tokens_bwd_kernel<T, 1, 4, ACT, GATE><<<grid, kThreads, shm, s>>>(a, p.lanes, p.gslots);
        else tokens_bwd_kernel<T, 1, 8, ACT, GATE><<<grid, kThreads, shm, s>>>(a, p.lanes, p.gslots);
    } else {
        const dim3 g1(p.blocks, a.N, (a.G + kThreads / 32 - 1) / (kThreads / 32));
        rows_part_kernel<T, true, ACT, GATE><<<g1, kThreads, 0, s>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        e = launch_dependent(rows_bwd_kernel<T, ACT, GATE>, dim3(p.blocks, a.N, (a.C + kThreads - 1) / kThreads),
                             kThreads, 0, s, a);
        if (e != cudaSuccess) return e;
    }
    if ((e = cudaGetLastError()) != cudaSuccess || !a.dweight) return e;
    return launch_dependent(wsum_kernel, dim3((2 * a.C + 31) / 32), 1024, 0, s, a);
}

template <typename T, bool BWD>
cudaError_t dispatch(const Args& a, const Plan& p, cudaStream_t s)
{
    auto go = [&](auto act, auto gate) {
        constexpr int A = decltype(act)::value;
        constexpr bool Z = decltype(gate)::value;
        if constexpr (BWD) return bwd_typed<T, A, Z>(a, p, s);
        else return fwd_typed<T, A, Z>(a, p, s);
    };
    using Silu = std::integral_constant<int, MDN_ACT_SILU>;
    using None = std::integral_constant<int, MDN_ACT_NONE>;
    if (a.act == MDN_ACT_SILU) return a.gate ? go(Silu{}, std::true_type{}) : go(Silu{}, std::false_type{});
    return a.gate ? go(None{}, std::true_type{}) : go(None{}, std::false_type{});
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool al_elem(const void* p, mdn_dtype dt)
{
    return (reinterpret_cast<uintptr_t>(p) & (dt == MDN_F32 ? 3u : 1u)) == 0;
}

mdn_status check(int N, int L, int C, int G, mdn_dtype dt, int act)
{
    if (N < 0 || L < 0 || C <= 0 || G <= 0 || C % G != 0) return MDN_ERR_INVALID_ARG;
    if (act != MDN_ACT_NONE && act != MDN_ACT_SILU) return MDN_ERR_INVALID_ARG;
    if (dt != MDN_F32 && dt != MDN_BF16) return MDN_ERR_UNSUPPORTED;
    // grid limits: rows and their groups per call, row blocks' second dimension
    if ((long long)N * G >= (1LL << 30) || C >= (1 << 22)) return MDN_ERR_UNSUPPORTED;
    if (L > 0x7fffff00) return MDN_ERR_UNSUPPORTED;  // row indices run a batch past L
    if (L > 1 && G > 8 * 65535) return MDN_ERR_UNSUPPORTED;  // 8 groups to a block of the rows form
    if (N > 65535) {  // only the tokens form takes more
        const Plan p = plan_of(N, L, C, G, dt == MDN_F32, true, true);
        const Plan q = plan_of(N, L, C, G, dt == MDN_F32, false, true);
        if (!p.tokens || !q.tokens) return MDN_ERR_UNSUPPORTED;
    }
    return MDN_OK;
}

}  // namespace
}  // namespace gn
}  // namespace mdn

using namespace mdn;

extern "C" {

size_t mdn_group_norm_workspace_size(int N, int L, int C, int G, mdn_dtype dtype, int backward)
{
    if (gn::check(N, L, C, G, dtype, MDN_ACT_NONE) != MDN_OK || N == 0 || L == 0) return 0;
    return gn::workspace_bytes(N, L, C, G, dtype == MDN_F32, backward != 0);
}

mdn_status mdn_group_norm_fwd(const void* x, const void* gate, mdn_dtype dtype, const float* weight,
                              const float* bias, int N, int L, int C, int G, float eps, int act,
                              void* y, float* mean, float* rstd, void* workspace, size_t ws_bytes,
                              mdn_stream_t stream)
{
    mdn_status st = gn::check(N, L, C, G, dtype, act);
    if (st != MDN_OK) return st;
    if (!(eps >= 0.f) || eps > 3.4e38f) return MDN_ERR_INVALID_ARG;
    if ((weight == nullptr) != (bias == nullptr)) return MDN_ERR_INVALID_ARG;
    if (N == 0 || L == 0) return MDN_OK;
    const void* tok[] = {x, y};
    for (const void* p : tok)
        if (!p || !gn::al_elem(p, dtype)) return MDN_ERR_INVALID_ARG;
    if (gate && !gn::al_elem(gate, dtype)) return MDN_ERR_INVALID_ARG;
    if (!mean || !rstd || !gn::al4(mean) || !gn::al4(rstd)) return MDN_ERR_INVALID_ARG;
    if (weight && (!gn::al4(weight) || !gn::al4(bias))) return MDN_ERR_INVALID_ARG;
    const bool vec = gn::al16(x) && gn::al16(y) && gn::al16(gate);
    const gn::Plan p = gn::plan_of(N, L, C, G, dtype == MDN_F32, vec, false);
    const size_t need = gn::workspace_bytes(N, L, C, G, dtype == MDN_F32, false);
    if (need && (!workspace || !gn::al16(workspace) || ws_bytes < need)) return MDN_ERR_INVALID_ARG;
    gn::Args a = {};
    a.x = x; a.gate = gate; a.weight = weight; a.bias = bias;
    a.N = N; a.L = L; a.C = C; a.G = G; a.eps = eps; a.act = act;
    a.y = y; a.mean = mean; a.rstd = rstd;
    a.part = static_cast<float*>(workspace);
    a.blocks = p.blocks;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == MDN_F32 ? gn::dispatch<float, false>(a, p, s)
                                           : gn::dispatch<__nv_bfloat16, false>(a, p, s);
    return e == cudaSuccess ? MDN_OK : cuda_fail(e);
}

mdn_status mdn_group_norm_bwd(const void* x, const void* gate, mdn_dtype dtype, const float* weight,
                              const float* bias, const float* mean, const float* rstd,
                              const void* dy, int N, int L, int C, int G, int act, void* dx,
                              void* dgate, float* dweight, float* dbias, void* workspace,
                              size_t ws_bytes, mdn_stream_t stream)
{
    mdn_status st = gn::check(N, L, C, G, dtype, act);
    if (st != MDN_OK) return st;
    if ((weight == nullptr) != (bias == nullptr)) return MDN_ERR_INVALID_ARG;
    if ((dweight == nullptr) != (dbias == nullptr) || (dweight && !weight)) return MDN_ERR_INVALID_ARG;
    if ((gate == nullptr) != (dgate == nullptr)) return MDN_ERR_INVALID_ARG;
    if (dweight && (!gn::al4(dweight) || !gn::al4(dbias))) return MDN_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0 || L == 0) {  // empty sums
        cudaError_t e = cudaSuccess;
        if (dweight) e = cudaMemsetAsync(dweight, 0, (size_t)C * sizeof(float), s);
        if (dweight && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, (size_t)C * sizeof(float), s);
        return e == cudaSuccess ? MDN_OK : cuda_fail(e);
    }
    const void* tok[] = {x, dy, dx};
    for (const void* p : tok)
        if (!p || !gn::al_elem(p, dtype)) return MDN_ERR_INVALID_ARG;
    if (gate && (!gn::al_elem(gate, dtype) || !gn::al_elem(dgate, dtype))) return MDN_ERR_INVALID_ARG;
    if (!mean || !rstd || !gn::al4(mean) || !gn::al4(rstd)) return MDN_ERR_INVALID_ARG;
    if (weight && (!gn::al4(weight) || !gn::al4(bias))) return MDN_ERR_INVALID_ARG;
    const bool vec = gn::al16(x) && gn::al16(dy) && gn::al16(dx) && gn::al16(gate) && gn::al16(dgate);
    const gn::Plan p = gn::plan_of(N, L, C, G, dtype == MDN_F32, vec, true);
    const size_t need = gn::workspace_bytes(N, L, C, G, dtype == MDN_F32, true);
    if (!workspace || !gn::al16(workspace) || ws_bytes < need) return MDN_ERR_INVALID_ARG;
    gn::Args a = {};
    a.x = x; a.gate = gate; a.weight = weight; a.bias = bias;
    a.N = N; a.L = L; a.C = C; a.G = G; a.act = act;
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.dy = dy; a.dx = dx; a.dgate = dgate; a.dweight = dweight; a.dbias = dbias;
    a.part = static_cast<float*>(workspace);
    a.wpart = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.part_bytes);
    a.blocks = p.blocks; a.prows = p.prows;
    const cudaError_t e = dtype == MDN_F32 ? gn::dispatch<float, true>(a, p, s)
                                           : gn::dispatch<__nv_bfloat16, true>(a, p, s);
    return e == cudaSuccess ? MDN_OK : cuda_fail(e);
}

}  // extern "C"
