// Internal declarations of the gated delta rule (see include/mdn.h,
// mdn_gdr_*).  Per (batch row or packed sequence, value head), with the state
// S of d x d entries (row index over the key, column index over the value):
//
//     vtilde_t = v_t - alpha_t S_{t-1}^T k_t
//     S_t      = alpha_t S_{t-1} + beta_t k_t vtilde_t^T
//     o_t      = scale S_t^T q_t
//
// and the adjoint that mdn_gdr_chunk_bwd runs from the saved vtilde (G_t is
// the adjoint of S_t):
//
//     dv_t = beta_t G_t^T k_t,            G_{t-1}' = alpha_t (G_t - k_t dv_t^T),
//     G_t  = scale q_t do_t^T + G_t',
//     dq_t = scale S_t do_t,              dk_t = beta_t G_t vtilde_t - alpha_t S_{t-1} dv_t,
//     dbeta_t = k_t^T G_t vtilde_t,       dalpha_log_t = alpha_t <G_t - k_t dv_t^T, S_{t-1}>.
//
// A key head serves H / Hk value heads; dq and dk are summed over them.
#pragma once

#include "mdn_internal.cuh"

namespace mdn {
namespace gdr {

// Everything a pass needs, with the workspace carved.  Token tensors are
// [rows, heads, D] with rows = B*T, or the packed tokens; nothing is padded
// or copied, a chain reads its own rows.
struct Args {
    const void* q;   // [rows, Hk, D]
    const void* k;
    const void* v;   // [rows, H, D]; backward: unused
    const float* alpha_log;  // [rows, H]
    const float* beta;
    float scale;
    const float* S0;         // [nseq, H, D, D] or null
    int B, T, Hk, H, D;      // packed: B = sequences, T = tokens of the buffer
    int NT;                  // chunks: per batch row, or of the whole packed call (upper bound)
    void* o;
    void* vt;                // forward: output, may be null; backward: input
    float* S_T;
    unsigned* status;        // [0] non-finite, [1] timeout, [2] bad cu_seqlens
    // packed sequences: checked offsets, chunk offsets and work order (device), else null
    const int* cu_s = nullptr;
    const int* cu_c = nullptr;
    const int* seq_order = nullptr;
    const int* chunk_order = nullptr;
    uint8_t* blk = nullptr;  // tensor-core path: operand blocks of every chunk and head
    unsigned* ready = nullptr;  // [chunks * H] block written, then the work counter and the number of
                                // operand CTAs without a limit; zeroed per call
    // backward
    const void* d_o = nullptr;
    const float* dS_T = nullptr;
    void* dq = nullptr;      // [rows, Hk, D], the inputs' type
    void* dk = nullptr;
    void* dv = nullptr;      // [rows, H, D]
    float* dalpha_log = nullptr;
    float* dbeta = nullptr;
    float* dS0 = nullptr;
    float* SS = nullptr;     // [chunks, H, D, D]  S entering each chunk
    float* GG = nullptr;     // [chunks, H, D, D]  adjoint of S leaving each chunk
    float* dvf = nullptr;    // [rows, H, D]  dv in fp32
    // backward on the tensor cores, per chunk and head (SL = d / ns column slices)
    int ns = 0;                      // columns per slice
    float* ssf = nullptr;            // [SL][16 warps][ns / 4][32]  entering state, in thread order
    __nv_bfloat16* sb = nullptr;     // [d, d]  entering state
    __nv_bfloat16* gb = nullptr;     // [d, d]  adjoint of the leaving state
    float* xs = nullptr;             // [SL][16 warps][ns / 32][32][4]  Diag(D) K S, in thread order
    float* po = nullptr;             // [SL][4][64]  scale D_r (S^T q_r) . do_r over 1/4 of the slice
    float* px = nullptr;             // [SL][4][64]  XS . dv
    float* pb = nullptr;             // [SL][4][64]  vtilde . dv / beta  (dbeta)
    float* pw = nullptr;             // [SL][4][64]  gam_r (G^T k_r) . vtilde_r
    float* gs = nullptr;             // [SL][16]  aC <G, S>
    __nv_bfloat16* dvl = nullptr;    // [rows, H, D]  dv - bf16(dv)
    float* dqp = nullptr;    // [rows, H, D]  dq, dk of each value head (H > Hk), else null
    float* dkp = nullptr;
};

// One chain: a state (batch row or sequence, value head) and its tokens.
struct Chain {
    long long state;  // index of the state, in units of D*D
    long long row0;   // first token row
    long long chunk0; // first chunk (index of the chunk buffers, times H plus h)
    int len, h, hk;
};

__device__ __forceinline__ Chain chain_of(const Args& a, long long c)
{
    Chain ch;
    ch.h = (int)(c % a.H);
    ch.hk = ch.h / (a.H / a.Hk);
    const long long r = c / a.H;
    if (a.cu_s) {
        const int seq = a.seq_order[r];
        ch.state = (long long)seq * a.H + ch.h;
        ch.row0 = a.cu_s[seq];
        ch.len = a.cu_s[seq + 1] - a.cu_s[seq];
        ch.chunk0 = a.cu_c[seq];
    } else {
        ch.state = c;
        ch.row0 = r * a.T;
        ch.len = a.T;
        ch.chunk0 = r * a.NT;
    }
    return ch;
}

// The tokens of chunk n of the call (of every head), or valid = 0 past the last.
struct ChunkRows {
    long long row0;
    int valid;
    bool first;  // the sequence's first chunk
};
__device__ __forceinline__ ChunkRows chunk_rows(const Args& a, long long n)
{
    ChunkRows c;
    int local, len;
    if (a.cu_s) {
        const int seq = varlen_seq_of_chunk(a.cu_c, a.B, (int)n);
        if (seq < 0) return ChunkRows{0, 0, false};
        local = (int)n - a.cu_c[seq];
        len = a.cu_s[seq + 1] - a.cu_s[seq];
        c.row0 = (long long)a.cu_s[seq] + (long long)local * kChunk;
    } else {
        local = (int)(n % a.NT);
        len = a.T;
        c.row0 = n / a.NT * a.T + (long long)local * kChunk;
    }
    const int rest = len - local * kChunk;
    c.valid = rest > kChunk ? kChunk : rest;
    c.first = local == 0;
    return c;
}

inline long long rows(const Args& a) { return a.cu_s ? a.T : (long long)a.B * a.T; }
inline long long chains(const Args& a) { return (long long)a.B * a.H; }
inline long long chunks(const Args& a) { return a.cu_s ? a.NT : (long long)a.B * a.NT; }

// Tensor-core path (bf16; backward d = 128).
cudaError_t launch_fwd_tc(const Args& a, cudaStream_t s);
cudaError_t launch_bwd_tc(const Args& a, cudaStream_t s);
// CUDA-core kernels, fp32 arithmetic, any supported type and d.
cudaError_t launch_fwd_simt(const Args& a, mdn_dtype dt, cudaStream_t s);
cudaError_t launch_bwd_simt(const Args& a, mdn_dtype dt, cudaStream_t s);
// Sums of dqp, dkp over the value heads of each key head, in head order.
cudaError_t launch_fold_heads(const Args& a, mdn_dtype dt, cudaStream_t s);
// One token; S_out may be S.
cudaError_t launch_step(const void* q, const void* k, const void* v, mdn_dtype dt,
                        const float* alpha_log, const float* beta, float scale, const float* S,
                        float* S_out, int B, int Hk, int H, int D, void* o, void* vt,
                        cudaStream_t s);

}  // namespace gdr
}  // namespace mdn
