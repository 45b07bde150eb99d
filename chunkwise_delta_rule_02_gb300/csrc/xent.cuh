// Shared by the linear softmax cross entropy's kernels (xent.cu on the tensor cores, xent_few.cu for few tokens).
#pragma once

#include "xent.h"

namespace gdn {
namespace xent {

using lay::ex2;
using lay::let_next_start;
using lay::wait_for_last;
using lay::kLog2e;

constexpr float kNone = -3.402823466e38f;   // maximum of no logits: the lowest number, so that differences to it are numbers or -infinity

// One product C = A B^T and how its tiles are cut: units of a tile and a part of the contraction.
struct Product {
    int M, N;                       // rows and columns of C that exist
    int mt, nt, kb;                 // tiles; 64-wide steps of the contraction
    int cuts, len;                  // parts of the contraction and their steps
    int b_row, b_k;                 // where B's rows and its contraction begin
    // OUT: the sum, where cuts > 1 of one part, [cuts][M][N] in `part`
    const float *add;               // [M][N] or null
    float *sum;                     // [M][N], or null: out
    float *part;
    void *out;
    long long out_b, out_t;         // row (b, t) of out at b out_b + t out_t
    long long pitch;                // the distance of rows where it is one, else 0
    int T, f32, wide;               // wide: out's float rows start at 16 bytes
    int out_box, sum_box;           // by tensor maps: out (bf16); sum, 1 stored, 2 added to what is there
};

struct Gemm {
    Product of[2];                  // the second of OUT only
    int seg;                        // SEG: steps of a segment, kSegment or kLongSegment
    int np;                         // plane products: nibbles of pa, pb
    uint32_t pa, pb;
    uint32_t *status;
    // STATS, GRAD, SCORE
    const int64_t *tgt;             // of token (b, t) at b tgt_b + t tgt_t
    const float *dloss;
    long long tgt_b, tgt_t, g_b, g_t, ignore;
    int T, V;
    const float *scale;             // the largest |dloss|, which D leaves out and the sums get back
    const float *lse;
    float *row;                     // [M] the target's logit
    float2 *part;
    int share;                      // SCORE: rows of w that a CTA has of a unit
    int v0, planes;
};

// A mean's dloss is one value for all tokens, whose rounding to bf16 would be off the same way in every row of D: up to 2^-8 of all
// gradients.  So D holds (exp(l - lse) - onehot) times dloss over its largest magnitude, and the sums are multiplied with that.
__device__ __forceinline__ float scale_of(const Gemm &p)
{
    const float s = *p.scale;
    return s > 0.f ? s : 1.f;
}

// A token's target, -1 for none: ignored, or (which the status word is told) outside the vocabulary.
__device__ __forceinline__ long long target_at(const Gemm &p, int row)
{
    return p.tgt[(long long)(row / p.T) * p.tgt_b + (long long)(row % p.T) * p.tgt_t];
}

__device__ __forceinline__ int target_from(const Gemm &p, long long v, bool tell)
{
    if (v == p.ignore) return -1;
    if (v >= 0 && v < p.V) return (int)v;
    if (tell) raise_status(p.status, kStatusBadOffsets);
    return -1;
}

__device__ __forceinline__ int target_of(const Gemm &p, int row, bool tell) { return target_from(p, target_at(p, row), tell); }

template <class K, class... A>
cudaError_t start(K kernel, long long blocks, int threads, int smem, cudaStream_t st, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaPeekAtLastError();
}

// What the kernels of a call have in common
Gemm common(const Call &c);
// loss and lse from P pieces a row (c.part)
cudaError_t join_rows(const Gemm &p, const Call &c, int P, cudaStream_t st);

}  // namespace xent
}  // namespace gdn
