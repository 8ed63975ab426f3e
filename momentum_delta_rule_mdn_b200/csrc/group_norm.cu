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
// Statistics are fp32 and never a difference of large sums: the tokens form
// takes the variance about the mean from registers, the rows form sums about
// each thread's first value and joins (count, mean, M2) triples.  dw and db are
// summed per thread, per block and then over blocks in a fixed order, so
// results do not depend on timing.
#include <algorithm>

#include "mdn_internal.cuh"

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
    int blocks;    // row blocks per n (rows form) / grid.x (tokens form, backward)
    int prows;     // partial rows of wpart
};

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }
__device__ __forceinline__ float act_of(float z, int act)
{
    return act == MDN_ACT_SILU ? z * sigmoid(z) : z;
}
// act(z) and its derivative
__device__ __forceinline__ void act_grad(float z, int act, float& f, float& df)
{
    f = z;
    df = 1.f;
    if (act == MDN_ACT_SILU) {
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
// VEC fp32 values that need only 4-byte alignment (weights)
template <int VEC>
__device__ __forceinline__ void ldw(const float* p, float* x)
{
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = p[e];
}

// Sum over `lanes` (a power of two) neighbouring lanes, in each of them.
__device__ __forceinline__ float sum_lanes(float x, int lanes)
{
    for (int off = 1; off < lanes; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// ---------------------------------------------------------------- tokens form (L = 1)
// `lanes` lanes per (token, group); NV vectors of VEC channels per lane.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kThreads) tokens_fwd_kernel(const Args a, int lanes)
{
    const int Cg = a.C / a.G, units = Cg / VEC;
    const int lane = threadIdx.x % lanes;
    const long long item = (long long)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
    const bool live = item < (long long)a.N * a.G;
    const int g = (int)(item % a.G);
    const size_t base = (size_t)item * Cg;
    const T* x = static_cast<const T*>(a.x) + base;
    float v[NV * VEC], z[NV * VEC];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = i * lanes + lane;
        if (live && u < units) {
            ldv<T, VEC>(x + u * VEC, v + i * VEC);
            if (a.gate) ldv<T, VEC>(static_cast<const T*>(a.gate) + base + u * VEC, z + i * VEC);
#pragma unroll
            for (int e = 0; e < VEC; ++e) s += v[i * VEC + e];
        }
    }
    const float mean = sum_lanes(s, lanes) / Cg;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (live && i * lanes + lane < units)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float d = v[i * VEC + e] - mean;
                q = fmaf(d, d, q);
            }
    const float rstd = 1.f / sqrtf(sum_lanes(q, lanes) / Cg + a.eps);
    if (!live) return;
    if (lane == 0) {
        a.mean[item] = mean;
        a.rstd[item] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = i * lanes + lane;
        if (u >= units) continue;
        float w[VEC], b[VEC], y[VEC];
        if (a.weight) {
            ldw<VEC>(a.weight + (size_t)g * Cg + u * VEC, w);
            ldw<VEC>(a.bias + (size_t)g * Cg + u * VEC, b);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float n = (v[i * VEC + e] - mean) * rstd;
            if (a.weight) n = fmaf(n, w[e], b[e]);
            y[e] = a.gate ? n * act_of(z[i * VEC + e], a.act) : act_of(n, a.act);
        }
        stv<T, VEC>(static_cast<T*>(a.y) + base + u * VEC, y);
    }
}

// One lane group per (group slot, token slot); a lane keeps its channels over
// all tokens it takes, so dw and db add up in registers.  grid.y tiles the
// groups, grid.x the tokens.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kThreads) tokens_bwd_kernel(const Args a, int lanes, int gslots)
{
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
    const int step = gridDim.x * per;
    for (int n0 = 0; n0 < a.N; n0 += step) {  // uniform trip count: shuffles below
        const int n = n0 + prow;
        const bool live = glive && n < a.N;
        const size_t base = ((size_t)n * a.G + g) * Cg;
        const float mean = live ? a.mean[(size_t)n * a.G + g] : 0.f;
        const float rstd = live ? a.rstd[(size_t)n * a.G + g] : 0.f;
        float xh[NV * VEC], dh[NV * VEC], z[NV * VEC];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int u = i * lanes + lane;
            if (live && u < units) {
                ldv<T, VEC>(static_cast<const T*>(a.x) + base + u * VEC, xh + i * VEC);
                ldv<T, VEC>(static_cast<const T*>(a.dy) + base + u * VEC, dh + i * VEC);
                if (a.gate) ldv<T, VEC>(static_cast<const T*>(a.gate) + base + u * VEC, z + i * VEC);
            }
        }
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
                act_grad(a.gate ? z[j] : nn, a.act, f, df);
                if (a.gate) {
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
            if (a.gate) stv<T, VEC>(static_cast<T*>(a.dgate) + base + u * VEC, dz);
        }
        const float m1 = sum_lanes(s1, lanes) / Cg, m2 = sum_lanes(s2, lanes) / Cg;
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
    if (!a.dweight || !glive) return;
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) {
        const int c = ((i / VEC) * lanes + lane) * VEC + i % VEC;
        if (c < Cg) {
            a.wpart[((size_t)prow * 2) * a.C + (size_t)g * Cg + c] = dw[i];
            a.wpart[((size_t)prow * 2 + 1) * a.C + (size_t)g * Cg + c] = db[i];
        }
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
template <typename T, bool BWD>
__global__ void __launch_bounds__(kThreads) rows_part_kernel(const Args a)
{
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
    float p = 0.f, q = 0.f;
    float* out = a.part + (((size_t)n * a.blocks + blockIdx.x) * a.G + g) * 2;
    if constexpr (!BWD) {
        const float shift = cnt > 0 ? ld_elem(x + base) : 0.f;  // the block's first value
        for (long long i = lane; i < cnt; i += 32) {
            const float d = ld_elem(x + base + (size_t)r * a.C + c) - shift;
            p += d;
            q = fmaf(d, d, q);
            r += sr; c += sc;
            if (c >= Cg) { c -= Cg; ++r; }
        }
        // (mean, M2) of the lane's values, joined pairwise over the lanes
        float k = (float)((cnt - lane + 31) / 32);
        if (cnt <= lane) k = 0.f;
        float mean = k > 0.f ? p / k : 0.f, m2 = k > 0.f ? q - p * mean : 0.f;
        for (int off = 1; off < 32; off <<= 1) {
            const float k2 = __shfl_xor_sync(0xffffffffu, k, off);
            const float e2 = __shfl_xor_sync(0xffffffffu, mean, off);
            const float q2 = __shfl_xor_sync(0xffffffffu, m2, off);
            const float t = k + k2, d = e2 - mean;
            if (t > 0.f) {
                const float f = k2 / t;
                m2 = m2 + q2 + d * d * k * f;
                mean = mean + d * f;
            }
            k = t;
        }
        if (lane == 0) {
            out[0] = mean + shift;
            out[1] = fmaxf(m2, 0.f);
        }
    } else {
        const T* dy = static_cast<const T*>(a.dy);
        const T* gate = static_cast<const T*>(a.gate);
        const float mean = a.mean[(size_t)n * a.G + g], rstd = a.rstd[(size_t)n * a.G + g];
        for (long long i = lane; i < cnt; i += 32) {
            const size_t at = base + (size_t)r * a.C + c;
            const float h = (ld_elem(x + at) - mean) * rstd;
            const float w = a.weight ? a.weight[(size_t)g * Cg + c] : 1.f;
            const float nn = a.weight ? fmaf(h, w, a.bias[(size_t)g * Cg + c]) : h;
            float f, df;
            act_grad(gate ? ld_elem(gate + at) : nn, a.act, f, df);
            const float dh = ld_elem(dy + at) * (gate ? f : df) * w;
            p += dh;
            q = fmaf(dh, h, q);
            r += sr; c += sc;
            if (c >= Cg) { c -= Cg; ++r; }
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
// shared memory; forward: mean and rstd, written out by the first row block.
template <bool BWD>
__device__ __forceinline__ void join_parts(const Args& a, int n, int g0, int g1, float2* st)
{
    const int Cg = a.C / a.G, per = (a.L + a.blocks - 1) / a.blocks;
    for (int g = g0 + (int)threadIdx.x; g < g1; g += kThreads) {
        const float* p = a.part + ((size_t)n * a.blocks * a.G + g) * 2;
        if constexpr (!BWD) {
            float k = 0.f, mean = 0.f, m2 = 0.f;
            for (int b = 0; b < a.blocks; ++b) {
                const int l0 = min(a.L, b * per), l1 = min(a.L, l0 + per);
                const float k2 = (float)(l1 - l0) * Cg;
                if (k2 <= 0.f) continue;
                const float d = p[(size_t)b * a.G * 2] - mean, t = k + k2, f = k2 / t;
                m2 += p[(size_t)b * a.G * 2 + 1] + d * d * k * f;
                mean += d * f;
                k = t;
            }
            const float rstd = 1.f / sqrtf(m2 / ((float)a.L * Cg) + a.eps);
            st[g - g0] = make_float2(mean, rstd);
            if (blockIdx.x == 0) {
                a.mean[(size_t)n * a.G + g] = mean;
                a.rstd[(size_t)n * a.G + g] = rstd;
            }
        } else {
            float s = 0.f, q = 0.f;
            for (int b = 0; b < a.blocks; ++b) {
                s += p[(size_t)b * a.G * 2];
                q += p[(size_t)b * a.G * 2 + 1];
            }
            const float m = (float)a.L * Cg;
            st[g - g0] = make_float2(s / m, q / m);
        }
    }
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) rows_fwd_kernel(const Args a)
{
    __shared__ float2 st[kThreads];  // a tile of kThreads channels touches at most as many groups
    const int Cg = a.C / a.G, n = blockIdx.y, c = blockIdx.z * kThreads + threadIdx.x;
    const int g0 = blockIdx.z * kThreads / Cg;
    const int g1 = (min(a.C, (int)(blockIdx.z + 1) * kThreads) - 1) / Cg + 1;
    join_parts<false>(a, n, g0, g1, st);
    if (c >= a.C) return;
    const RowBlock rb = row_block(a);
    const float2 ms = st[c / Cg - g0];
    const float w = a.weight ? a.weight[c] : 1.f, b = a.weight ? a.bias[c] : 0.f;
    const T* gate = static_cast<const T*>(a.gate);
    size_t at = ((size_t)n * a.L + rb.l0) * a.C + c;
    for (int l = rb.l0; l < rb.l1; ++l, at += a.C) {
        const float nn = fmaf((ld_elem(static_cast<const T*>(a.x) + at) - ms.x) * ms.y, w, b);
        st_elem(static_cast<T*>(a.y) + at,
                gate ? nn * act_of(ld_elem(gate + at), a.act) : act_of(nn, a.act));
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) rows_bwd_kernel(const Args a)
{
    __shared__ float2 st[kThreads];
    const int Cg = a.C / a.G, n = blockIdx.y, c = blockIdx.z * kThreads + threadIdx.x;
    const int g0 = blockIdx.z * kThreads / Cg;
    const int g1 = (min(a.C, (int)(blockIdx.z + 1) * kThreads) - 1) / Cg + 1;
    join_parts<true>(a, n, g0, g1, st);
    if (c >= a.C) return;
    const RowBlock rb = row_block(a);
    const int g = c / Cg;
    const float2 m = st[g - g0];
    const float mean = a.mean[(size_t)n * a.G + g], rstd = a.rstd[(size_t)n * a.G + g];
    const float w = a.weight ? a.weight[c] : 1.f, b = a.weight ? a.bias[c] : 0.f;
    const T* gate = static_cast<const T*>(a.gate);
    float dw = 0.f, db = 0.f;
    size_t at = ((size_t)n * a.L + rb.l0) * a.C + c;
    for (int l = rb.l0; l < rb.l1; ++l, at += a.C) {
        const float h = (ld_elem(static_cast<const T*>(a.x) + at) - mean) * rstd;
        const float nn = fmaf(h, w, b), dy = ld_elem(static_cast<const T*>(a.dy) + at);
        float f, df;
        act_grad(gate ? ld_elem(gate + at) : nn, a.act, f, df);
        const float dn = dy * (gate ? f : df);
        if (gate) st_elem(static_cast<T*>(a.dgate) + at, dy * nn * df);
        dw = fmaf(dn, h, dw);
        db += dn;
        st_elem(static_cast<T*>(a.dx) + at, rstd * (dn * w - m.x - h * m.y));
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
    if (c < 2LL * a.C)
        for (int r = r0; r < a.prows; r += 32) s += a.wpart[(size_t)r * 2 * a.C + c];
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
    int gslots;   // backward, tokens form
    int blocks;   // row blocks per n (rows), or token blocks (backward, tokens form)
    int gtiles;   // backward, tokens form
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
        if (bwd) {
            const int slots = kThreads / p.lanes;
            p.gslots = 1;
            while (p.gslots < slots && p.gslots < G) p.gslots <<= 1;
            p.gtiles = (G + p.gslots - 1) / p.gslots;
            const int per = slots / p.gslots;
            const int most = (N + per - 1) / per;
            p.blocks = std::max(1, std::min(most, want / p.gtiles));
            p.prows = p.blocks * per;
        }
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

template <typename T>
cudaError_t fwd_typed(const Args& a0, const Plan& p, cudaStream_t s)
{
    Args a = a0;
    constexpr int V = 16 / (int)sizeof(T);
    ProfScope ps(kGroupNorm, s);
    if (p.tokens) {
        const int per = kThreads / p.lanes;
        const long long items = (long long)a.N * a.G;
        const unsigned grid = (unsigned)((items + per - 1) / per);
        if (p.vec && p.nv == 1) tokens_fwd_kernel<T, V, 1><<<grid, kThreads, 0, s>>>(a, p.lanes);
        else if (p.vec) tokens_fwd_kernel<T, V, 2><<<grid, kThreads, 0, s>>>(a, p.lanes);
        else if (p.nv == 4) tokens_fwd_kernel<T, 1, 4><<<grid, kThreads, 0, s>>>(a, p.lanes);
        else tokens_fwd_kernel<T, 1, 8><<<grid, kThreads, 0, s>>>(a, p.lanes);
        return cudaGetLastError();
    }
    const dim3 g1(p.blocks, a.N, (a.G + kThreads / 32 - 1) / (kThreads / 32));
    rows_part_kernel<T, false><<<g1, kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    rows_fwd_kernel<T><<<dim3(p.blocks, a.N, (a.C + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_typed(const Args& a0, const Plan& p, cudaStream_t s)
{
    Args a = a0;
    constexpr int V = 16 / (int)sizeof(T);
    ProfScope ps(kGroupNormBwd, s);
    cudaError_t e;
    if (p.tokens) {
        const dim3 grid(p.blocks, p.gtiles);
        if (p.vec && p.nv == 1) tokens_bwd_kernel<T, V, 1><<<grid, kThreads, 0, s>>>(a, p.lanes, p.gslots);
        else if (p.vec) tokens_bwd_kernel<T, V, 2><<<grid, kThreads, 0, s>>>(a, p.lanes, p.gslots);
        else if (p.nv == 4) tokens_bwd_kernel<T, 1, 4><<<grid, kThreads, 0, s>>>(a, p.lanes, p.gslots);
        else tokens_bwd_kernel<T, 1, 8><<<grid, kThreads, 0, s>>>(a, p.lanes, p.gslots);
    } else {
        const dim3 g1(p.blocks, a.N, (a.G + kThreads / 32 - 1) / (kThreads / 32));
        rows_part_kernel<T, true><<<g1, kThreads, 0, s>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        rows_bwd_kernel<T><<<dim3(p.blocks, a.N, (a.C + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
    }
    if ((e = cudaGetLastError()) != cudaSuccess || !a.dweight) return e;
    wsum_kernel<<<(2 * a.C + 31) / 32, 1024, 0, s>>>(a);
    return cudaGetLastError();
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
    const cudaError_t e = dtype == MDN_F32 ? gn::fwd_typed<float>(a, p, s)
                                           : gn::fwd_typed<__nv_bfloat16>(a, p, s);
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
    const cudaError_t e = dtype == MDN_F32 ? gn::bwd_typed<float>(a, p, s)
                                           : gn::bwd_typed<__nv_bfloat16>(a, p, s);
    return e == cudaSuccess ? MDN_OK : cuda_fail(e);
}

}  // extern "C"
