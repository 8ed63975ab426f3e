// The C entry points of the gated delta rule (include/mdn.h, mdn_gdr_*):
// argument validation, workspace layout and kernel dispatch.
#include <cmath>

#include "gdr_tc.cuh"

using namespace mdn;

namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned_elem(const void* p, mdn_dtype dt)
{
    return (reinterpret_cast<uintptr_t>(p) & (dt == MDN_F32 ? 3u : 1u)) == 0;
}

// One call's sizes.  packed: B = sequences, T = tokens of the packed buffer.
struct Sizes {
    int B, T, Hk, H, dk, dv, C;
    mdn_dtype dt;
    bool packed;
    int flags;
    // On the tensor cores?  Sequences of less than a chunk or so are cheaper token by token (and
    // exact in fp32).  Measured, one and 1024 chains of d 128, tensor cores and CUDA cores, us:
    // forward 16 tokens 25 and 10, 131 and 84; 32: 23 and 13, 133 and 144; 64: 21 and 18, 136
    // and 264; backward 16 tokens 48 and 40, 307 and 289; 32: 48 and 64, 311 and 491.  Forward,
    // d 64, 64 tokens: 21 and 16, 105 and 90.  Of a packed call only the sum is known.
    bool bf16() const { return dt == MDN_BF16 && !(flags & MDN_FORCE_SIMT); }
    bool tc(bool bwd) const { return bf16() && (bwd ? dk == 128 && T > 16 : T > 4096 / dk); }
    long long rows() const { return packed ? T : (long long)B * T; }
    // chunks of the call: every sequence ends in at most one partial chunk
    long long chunks() const
    {
        return packed ? (long long)T / C + B : (long long)B * (((long long)T + C - 1) / C);
    }
};

mdn_status check_sizes(const Sizes& z)
{
    if (z.B < 0 || z.T < 0 || z.H < 0 || z.Hk < 0 || z.dk <= 0 || z.dv <= 0 || z.C <= 0)
        return MDN_ERR_INVALID_ARG;
    if (z.H > 0 && (z.Hk == 0 || z.H % z.Hk != 0)) return MDN_ERR_INVALID_ARG;
    if (z.dt != MDN_F32 && z.dt != MDN_BF16) return MDN_ERR_UNSUPPORTED;
    if (z.dk != z.dv || (z.dk != 64 && z.dk != 128) || z.C != kChunk) return MDN_ERR_UNSUPPORTED;
    // grids and 32-bit chunk indices
    if (z.chunks() * z.H >= (1LL << 31) || (long long)z.B * z.H >= (1LL << 31) / 4 ||
        z.chunks() * z.C >= (1LL << 31))
        return MDN_ERR_UNSUPPORTED;
    return MDN_OK;
}

struct Layout {
    size_t status, head, cu_s, cu_c, seq_order, chunk_order;
    size_t blk;                    // forward on the tensor cores
    size_t SS, GG, dvf, dqp, dkp;  // backward on CUDA cores
    size_t ssf, sb, gb, xs, po, px, pb, pw, gs, dvl;  // backward on the tensor cores
    int ns;
    size_t total;
};

Layout layout(const Sizes& z, bool bwd)
{
    Layout w = {};
    // status words first (mdn_chunk_fwd_status reads them there), then the ready flags and the
    // work counter of the operand blocks: one memset clears both
    size_t off = 64;
    if (z.tc(bwd)) off += ((size_t)z.chunks() * z.H + 2) * sizeof(unsigned);
    w.head = off;
    off = align_up(off);
    if (z.packed) {
        w.cu_s = off;        off += align_up((size_t)(z.B + 1) * sizeof(int));
        w.cu_c = off;        off += align_up((size_t)(z.B + 1) * sizeof(int));
        w.seq_order = off;   off += align_up((size_t)z.B * sizeof(int));
        w.chunk_order = off; off += align_up((size_t)z.chunks() * sizeof(int));
    }
    if (!bwd && z.tc(false)) {
        w.blk = off; off += align_up((size_t)z.chunks() * z.H * gdr::kBlkBytes);
    }
    if (bwd && z.tc(true)) {
        const size_t ch = (size_t)z.chunks() * z.H, dd = (size_t)z.dk * z.dv;
        // 32 columns a slice while four CTAs per chain fit a B200's 148 SMs at once (the
        // shortest chunk step), else 64 (half the loads of K, Q and the images)
        w.ns = (long long)z.B * z.H * 4 <= 148 ? 32 : 64;
        const size_t sl = z.dk / w.ns;
        w.blk = off; off += align_up(ch * gdr::kBwdBytes);
        w.ssf = off; off += align_up(ch * dd * sizeof(float));
        w.sb = off;  off += align_up(ch * dd * 2);
        w.gb = off;  off += align_up(ch * dd * 2);
        w.xs = off;  off += align_up(ch * kChunk * z.dk * sizeof(float));
        w.po = off;  off += align_up(ch * sl * 4 * kChunk * sizeof(float));
        w.px = off;  off += align_up(ch * sl * 4 * kChunk * sizeof(float));
        w.pb = off;  off += align_up(ch * sl * 4 * kChunk * sizeof(float));
        w.pw = off;  off += align_up(ch * sl * 4 * kChunk * sizeof(float));
        w.gs = off;  off += align_up(ch * sl * 16 * sizeof(float));
        w.dvl = off; off += align_up((size_t)z.rows() * z.H * z.dk * 2);
    } else if (bwd) {
        const size_t states = (size_t)z.chunks() * z.H * z.dk * z.dv * sizeof(float);
        const size_t tok = (size_t)z.rows() * z.H * z.dk * sizeof(float);
        w.SS = off;  off += align_up(states);
        w.GG = off;  off += align_up(states);
        w.dvf = off; off += align_up(tok);
        if (z.H > z.Hk) {
            w.dqp = off; off += align_up(tok);
            w.dkp = off; off += align_up(tok);
        }
    }
    w.total = off;
    return w;
}

size_t ws_size(const Sizes& z, bool bwd)
{
    return check_sizes(z) == MDN_OK ? layout(z, bwd).total : 0;
}

// Clears the status words and, for packed sequences, checks the offsets.
mdn_status begin(gdr::Args& a, const Sizes& z, const Layout& w, char* ws, const int* cu_seqlens,
                 cudaStream_t s)
{
    a.B = z.B; a.T = z.T; a.Hk = z.Hk; a.H = z.H; a.D = z.dk;
    a.NT = (int)(z.packed ? z.chunks() : ((long long)z.T + z.C - 1) / z.C);
    a.status = reinterpret_cast<unsigned*>(ws + w.status);
    if (w.head > 64) a.ready = a.status + 16;
    cudaError_t e = cudaMemsetAsync(a.status, 0, w.head, s);
    if (e != cudaSuccess) return cuda_fail(e);
    if (!z.packed) return MDN_OK;
    int* cu_s = reinterpret_cast<int*>(ws + w.cu_s);
    int* cu_c = reinterpret_cast<int*>(ws + w.cu_c);
    int* seq = reinterpret_cast<int*>(ws + w.seq_order);
    e = launch_varlen_setup(cu_seqlens, z.B, z.T, a.NT, cu_s, cu_c, seq,
                            reinterpret_cast<int*>(ws + w.chunk_order), a.status + 2, s,
                            /*exact=*/false);
    if (e != cudaSuccess) return cuda_fail(e);
    a.cu_s = cu_s; a.cu_c = cu_c; a.seq_order = seq;
    a.chunk_order = reinterpret_cast<int*>(ws + w.chunk_order);
    return MDN_OK;
}

// MDN_ZERO_BEHIND: zeros in the rows of packed outputs behind the last sequence.
struct Rest {
    static constexpr int kMost = 5;
    void* p[kMost];
    size_t row_bytes[kMost];  // multiples of 4
    int n;
};

__global__ void __launch_bounds__(256) zero_behind_kernel(const Rest r, const int* cu_s, int B, int total)
{
    const size_t rows = (size_t)(total - cu_s[B]), step = (size_t)gridDim.x * 256;
    const size_t tid = (size_t)blockIdx.x * 256 + threadIdx.x;
    for (int i = 0; i < r.n; ++i) {
        char* p = static_cast<char*>(r.p[i]) + (size_t)cu_s[B] * r.row_bytes[i];
        const size_t bytes = rows * r.row_bytes[i];
        if (r.row_bytes[i] % 16 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
            for (size_t e = tid; e < bytes / 16; e += step) reinterpret_cast<uint4*>(p)[e] = make_uint4(0, 0, 0, 0);
        } else {
            for (size_t e = tid; e < bytes / 4; e += step) reinterpret_cast<unsigned*>(p)[e] = 0u;
        }
    }
}

// cu_s: the checked offsets, or null (no sequences: every row is behind).
mdn_status zero_behind(const Rest& r, const int* cu_s, const Sizes& z, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    if (z.T == 0) return MDN_OK;
    for (int i = 0; i < r.n && !cu_s; ++i) {
        if (!r.p[i]) return MDN_ERR_INVALID_ARG;
        if (e == cudaSuccess) e = cudaMemsetAsync(r.p[i], 0, (size_t)z.T * r.row_bytes[i], s);
    }
    if (cu_s) {
        zero_behind_kernel<<<148 * 2, 256, 0, s>>>(r, cu_s, z.B, z.T);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? MDN_OK : cuda_fail(e);
}

bool bad_flags(const Sizes& z, int flags)
{
    return flags & ~(MDN_CHECK_FINITE | MDN_FORCE_SIMT | (z.packed ? MDN_ZERO_BEHIND : 0));
}

struct Out {
    const void* p;
    size_t n;
    bool bf16;
};

// MDN_CHECK_FINITE: scan the outputs, synchronise and report.
mdn_status report(const Out* outs, int n, unsigned* status, cudaStream_t s)
{
    cudaError_t e;
    for (int i = 0; i < n; ++i)
        if (outs[i].p && (e = launch_finite_check(outs[i].p, outs[i].n, outs[i].bf16, status, s)))
            return cuda_fail(e);
    unsigned host[3] = {0, 0, 0};
    if ((e = cudaMemcpyAsync(host, status, sizeof(host), cudaMemcpyDeviceToHost, s))) return cuda_fail(e);
    if ((e = cudaStreamSynchronize(s))) return cuda_fail(e);
    if (host[2]) return MDN_ERR_INVALID_ARG;
    if (host[1]) return MDN_ERR_TIMEOUT;
    return host[0] ? MDN_ERR_NONFINITE : MDN_OK;
}

mdn_status fwd_impl(const Sizes& z, const void* q, const void* k, const void* v,
                    const float* alpha_log, const float* beta, float scale, const int* cu_seqlens,
                    const float* S0, void* o, void* vtilde, float* S_T, void* workspace,
                    size_t ws_bytes, int flags, mdn_stream_t stream)
{
    mdn_status st = check_sizes(z);
    if (st != MDN_OK) return st;
    if (bad_flags(z, flags)) return MDN_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return MDN_ERR_INVALID_ARG;
    const size_t row = (size_t)z.H * z.dk * (z.dt == MDN_BF16 ? 2 : 4);
    const Rest rest = {{o, vtilde}, {row, row}, vtilde ? 2 : 1};
    if (z.B == 0 && z.H > 0 && (flags & MDN_ZERO_BEHIND))
        return zero_behind(rest, nullptr, z, reinterpret_cast<cudaStream_t>(stream));
    if (z.B == 0 || z.H == 0) return MDN_OK;
    if (z.packed && (!cu_seqlens || !aligned4(cu_seqlens))) return MDN_ERR_INVALID_ARG;
    if (!S_T || !aligned16(S_T) || !aligned16(S0)) return MDN_ERR_INVALID_ARG;
    if (z.rows() > 0) {
        const void* tok[] = {q, k, v, o};
        for (const void* p : tok)
            if (!p || !aligned16(p)) return MDN_ERR_INVALID_ARG;
        if (!aligned16(vtilde)) return MDN_ERR_INVALID_ARG;
        if (!alpha_log || !beta || !aligned4(alpha_log) || !aligned4(beta)) return MDN_ERR_INVALID_ARG;
    }
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % kAlign) return MDN_ERR_INVALID_ARG;
    const Layout w = layout(z, false);
    if (ws_bytes < w.total) return MDN_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    gdr::Args a;
    a.q = q; a.k = k; a.v = v; a.alpha_log = alpha_log; a.beta = beta; a.scale = scale; a.S0 = S0;
    a.o = o; a.vt = vtilde; a.S_T = S_T;
    if (w.blk) a.blk = reinterpret_cast<uint8_t*>(ws + w.blk);
    if ((st = begin(a, z, w, ws, cu_seqlens, s)) != MDN_OK) return st;
    if ((flags & MDN_ZERO_BEHIND) && (st = zero_behind(rest, a.cu_s, z, s)) != MDN_OK) return st;
    // no tokens: S_T = S0, which the CUDA-core kernel's walk over nothing gives
    const cudaError_t e = z.tc(false) ? gdr::launch_fwd_tc(a, s) : gdr::launch_fwd_simt(a, z.dt, s);
    if (e != cudaSuccess) return cuda_fail(e);
    if (!(flags & MDN_CHECK_FINITE)) return MDN_OK;
    const bool bf = z.dt == MDN_BF16;
    const size_t tok = (size_t)z.rows() * z.H * z.dk, sta = (size_t)z.B * z.H * z.dk * z.dv;
    // a packed buffer may have rows behind its last sequence, which the pass does not write
    const Out outs[] = {{z.packed ? nullptr : o, tok, bf}, {z.packed ? nullptr : vtilde, tok, bf},
                        {S_T, sta, false}};
    return report(outs, 3, a.status, s);
}

mdn_status bwd_impl(const Sizes& z, const void* q, const void* k, const float* alpha_log,
                    const float* beta, float scale, const int* cu_seqlens, const float* S0,
                    const void* vtilde, const void* d_o, const float* dS_T, void* dq, void* dk_out,
                    void* dv_out, float* dalpha_log, float* dbeta, float* dS0, void* workspace,
                    size_t ws_bytes, int flags, mdn_stream_t stream)
{
    mdn_status st = check_sizes(z);
    if (st != MDN_OK) return st;
    if (bad_flags(z, flags)) return MDN_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return MDN_ERR_INVALID_ARG;
    const size_t el = z.dt == MDN_BF16 ? 2 : 4, krow = z.Hk * z.dk * el, gate = (size_t)z.H * 4;
    const Rest rest = {{dq, dk_out, dv_out, dalpha_log, dbeta}, {krow, krow, z.H * z.dk * el, gate, gate}, 5};
    if (z.B == 0 && z.H > 0 && (flags & MDN_ZERO_BEHIND))
        return zero_behind(rest, nullptr, z, reinterpret_cast<cudaStream_t>(stream));
    if (z.B == 0 || z.H == 0) return MDN_OK;
    if (z.packed && (!cu_seqlens || !aligned4(cu_seqlens))) return MDN_ERR_INVALID_ARG;
    if (!dS0 || !aligned16(dS0) || !aligned16(dS_T) || !aligned16(S0)) return MDN_ERR_INVALID_ARG;
    if (z.rows() > 0) {
        const void* tok[] = {q, k, vtilde, d_o, dq, dk_out, dv_out};
        for (const void* p : tok)
            if (!p || !aligned16(p)) return MDN_ERR_INVALID_ARG;
        const void* g[] = {alpha_log, beta, dalpha_log, dbeta};
        for (const void* p : g)
            if (!p || !aligned4(p)) return MDN_ERR_INVALID_ARG;
    }
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % kAlign) return MDN_ERR_INVALID_ARG;
    const Layout w = layout(z, true);
    if (ws_bytes < w.total) return MDN_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    gdr::Args a;
    a.q = q; a.k = k; a.v = nullptr; a.alpha_log = alpha_log; a.beta = beta; a.scale = scale; a.S0 = S0;
    a.o = nullptr; a.vt = const_cast<void*>(vtilde); a.S_T = nullptr;
    a.d_o = d_o; a.dS_T = dS_T; a.dq = dq; a.dk = dk_out; a.dv = dv_out;
    a.dalpha_log = dalpha_log; a.dbeta = dbeta; a.dS0 = dS0;
    auto at = [&](size_t o) { return o ? reinterpret_cast<float*>(ws + o) : nullptr; };
    a.SS = at(w.SS); a.GG = at(w.GG); a.dvf = at(w.dvf); a.dqp = at(w.dqp); a.dkp = at(w.dkp);
    a.ns = w.ns;
    a.blk = reinterpret_cast<uint8_t*>(at(w.blk));
    a.ssf = at(w.ssf); a.xs = at(w.xs); a.po = at(w.po); a.px = at(w.px); a.pb = at(w.pb);
    a.pw = at(w.pw); a.gs = at(w.gs);
    a.sb = reinterpret_cast<__nv_bfloat16*>(at(w.sb));
    a.gb = reinterpret_cast<__nv_bfloat16*>(at(w.gb));
    a.dvl = reinterpret_cast<__nv_bfloat16*>(at(w.dvl));
    if ((st = begin(a, z, w, ws, cu_seqlens, s)) != MDN_OK) return st;
    if ((flags & MDN_ZERO_BEHIND) && (st = zero_behind(rest, a.cu_s, z, s)) != MDN_OK) return st;
    // no tokens: dS0 = dS_T, which the CUDA-core chain's walk over nothing gives
    const bool tc = z.tc(true);
    cudaError_t e = tc ? gdr::launch_bwd_tc(a, s) : gdr::launch_bwd_simt(a, z.dt, s);
    if (e == cudaSuccess && a.dqp) e = gdr::launch_fold_heads(a, z.dt, s);
    if (e != cudaSuccess) return cuda_fail(e);
    if (!(flags & MDN_CHECK_FINITE)) return MDN_OK;
    const bool bf = z.dt == MDN_BF16;
    const size_t tok = (size_t)z.rows() * z.H, key = (size_t)z.rows() * z.Hk * z.dk;
    const bool whole = !z.packed;  // as in the forward pass
    const Out outs[] = {{whole ? dq : nullptr, key, bf}, {whole ? dk_out : nullptr, key, bf},
                        {whole ? dv_out : nullptr, tok * z.dk, bf},
                        {whole ? dalpha_log : nullptr, tok, false}, {whole ? dbeta : nullptr, tok, false},
                        {dS0, (size_t)z.B * z.H * z.dk * z.dv, false}};
    return report(outs, 6, a.status, s);
}

}  // namespace

extern "C" {

size_t mdn_gdr_chunk_fwd_workspace_size(int B, int T, int Hk, int H, int dk, int dv, int C,
                                        mdn_dtype in_dtype, int flags)
{
    return ws_size(Sizes{B, T, Hk, H, dk, dv, C, in_dtype, false, flags}, false);
}

size_t mdn_gdr_chunk_fwd_varlen_workspace_size(int N, int total_T, int Hk, int H, int dk, int dv,
                                               int C, mdn_dtype in_dtype, int flags)
{
    return ws_size(Sizes{N, total_T, Hk, H, dk, dv, C, in_dtype, true, flags}, false);
}

size_t mdn_gdr_chunk_bwd_workspace_size(int B, int T, int Hk, int H, int dk, int dv, int C,
                                        mdn_dtype in_dtype, int flags)
{
    return ws_size(Sizes{B, T, Hk, H, dk, dv, C, in_dtype, false, flags}, true);
}

size_t mdn_gdr_chunk_bwd_varlen_workspace_size(int N, int total_T, int Hk, int H, int dk, int dv,
                                               int C, mdn_dtype in_dtype, int flags)
{
    return ws_size(Sizes{N, total_T, Hk, H, dk, dv, C, in_dtype, true, flags}, true);
}

mdn_status mdn_gdr_chunk_fwd(const void* q, const void* k, const void* v, mdn_dtype in_dtype,
                             const float* alpha_log, const float* beta, float scale,
                             const float* S0, int B, int T, int Hk, int H, int dk, int dv, int C,
                             void* o, void* vtilde, float* S_T, void* workspace, size_t ws_bytes,
                             int flags, mdn_stream_t stream)
{
    return fwd_impl(Sizes{B, T, Hk, H, dk, dv, C, in_dtype, false, flags}, q, k, v, alpha_log, beta,
                    scale, nullptr, S0, o, vtilde, S_T, workspace, ws_bytes, flags, stream);
}

mdn_status mdn_gdr_chunk_fwd_varlen(const void* q, const void* k, const void* v,
                                    mdn_dtype in_dtype, const float* alpha_log, const float* beta,
                                    float scale, const int* cu_seqlens, int N, int total_T,
                                    const float* S0, int Hk, int H, int dk, int dv, int C, void* o,
                                    void* vtilde, float* S_T, void* workspace, size_t ws_bytes,
                                    int flags, mdn_stream_t stream)
{
    return fwd_impl(Sizes{N, total_T, Hk, H, dk, dv, C, in_dtype, true, flags}, q, k, v, alpha_log, beta,
                    scale, cu_seqlens, S0, o, vtilde, S_T, workspace, ws_bytes, flags, stream);
}

mdn_status mdn_gdr_chunk_bwd(const void* q, const void* k, mdn_dtype in_dtype,
                             const float* alpha_log, const float* beta, float scale,
                             const float* S0, const void* vtilde, const void* d_o,
                             const float* dS_T, int B, int T, int Hk, int H, int dk, int dv, int C,
                             void* dq, void* dk_out, void* dv_out, float* dalpha_log, float* dbeta,
                             float* dS0, void* workspace, size_t ws_bytes, int flags,
                             mdn_stream_t stream)
{
    return bwd_impl(Sizes{B, T, Hk, H, dk, dv, C, in_dtype, false, flags}, q, k, alpha_log, beta, scale,
                    nullptr, S0, vtilde, d_o, dS_T, dq, dk_out, dv_out, dalpha_log, dbeta, dS0,
                    workspace, ws_bytes, flags, stream);
}

mdn_status mdn_gdr_chunk_bwd_varlen(const void* q, const void* k, mdn_dtype in_dtype,
                                    const float* alpha_log, const float* beta, float scale,
                                    const int* cu_seqlens, int N, int total_T, const float* S0,
                                    const void* vtilde, const void* d_o, const float* dS_T, int Hk,
                                    int H, int dk, int dv, int C, void* dq, void* dk_out,
                                    void* dv_out, float* dalpha_log, float* dbeta, float* dS0,
                                    void* workspace, size_t ws_bytes, int flags,
                                    mdn_stream_t stream)
{
    return bwd_impl(Sizes{N, total_T, Hk, H, dk, dv, C, in_dtype, true, flags}, q, k, alpha_log, beta,
                    scale, cu_seqlens, S0, vtilde, d_o, dS_T, dq, dk_out, dv_out, dalpha_log,
                    dbeta, dS0, workspace, ws_bytes, flags, stream);
}

mdn_status mdn_gdr_step(const void* q, const void* k, const void* v, mdn_dtype in_dtype,
                        const float* alpha_log, const float* beta, float scale, const float* S,
                        float* S_out, int B, int Hk, int H, int dk, int dv, void* o, void* vtilde,
                        int flags, mdn_stream_t stream)
{
    mdn_status st = check_sizes(Sizes{B, 1, Hk, H, dk, dv, kChunk, in_dtype, false, 0});
    if (st != MDN_OK) return st;
    if (flags != 0 || !std::isfinite(scale)) return MDN_ERR_INVALID_ARG;
    if (B == 0 || H == 0) return MDN_OK;
    const void* tok[] = {q, k, v, o};
    for (const void* p : tok)
        if (!p || !aligned_elem(p, in_dtype)) return MDN_ERR_INVALID_ARG;
    if (vtilde && !aligned_elem(vtilde, in_dtype)) return MDN_ERR_INVALID_ARG;
    if (!alpha_log || !beta || !aligned4(alpha_log) || !aligned4(beta)) return MDN_ERR_INVALID_ARG;
    if (!S || !S_out || !aligned16(S) || !aligned16(S_out)) return MDN_ERR_INVALID_ARG;
    const cudaError_t e = gdr::launch_step(q, k, v, in_dtype, alpha_log, beta, scale, S, S_out, B,
                                           Hk, H, dk, o, vtilde,
                                           reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MDN_OK : cuda_fail(e);
}

}  // extern "C"
