// Launchers of the linear softmax cross entropy, called by xent_api.cu with checked arguments.
#pragma once

#include "layers.h"

namespace gdn {
namespace xent {

// An operand matrix as the tensor maps take it: bf16 [planes][rows][pitch]
struct Operand {
    const void *p;
    long long pitch, plane;         // elements
};

// A launch's sizes.  M tokens, K features, V vocabulary entries; float32 inputs are held as
// three bf16 planes (x = x0 + x1 + x2), bf16 ones as one.
struct Call {
    const dn_xent_shape *s;
    const dn_view *x, *w, *targets, *dloss, *dx;
    int M, K, V, planes;
    int piece;                      // vocabulary entries of a piece (backward)
    Operand xo, wo;
    bool pack_x, pack_w;
    bool few;                       // few tokens: without the tensor cores, x and w read in place
    uint32_t *status;
    float *row;                     // forward: [M] the target's logit
    float2 *part;                   // forward: [parts_of][M] maximum and sum
    char *d;                        // backward: [planes][M][piece] bf16 gradients of the logits of a piece
    float *acc;                     // backward: [M][K] sums of dx over pieces (more than one)
    float *cut;                     // backward: parts of dx and of a piece of dw whose contractions are cut
    void *dx_rows, *dw_rows;        // backward, bf16 of a width that is no multiple of 8: results in rows that start at 16 bytes
    float *loss, *lse;
    void *dw;
};

int tiles_of(int n);                // of 256
// Rows of a copy start at the 32 bytes that the L2 cache moves (5082 tokens of 57991 x 147, backward, with 16 and 32: 558 and 520 us)
inline long long copy_pitch(long long K) { return (K + 15) / 16 * 16; }
int parts_of(int M, int V);
// Whether a call goes without the tensor cores, and its blocks (rows of `part`, parts of dx)
bool few_tokens(int M, int K, bool f32);
int few_blocks(int M, int K, int V, bool bwd);
void cuts_of(int M, int K, int n, int planes, int &dx, int &dw);   // parts that a piece's two contractions are cut into
cudaError_t few_forward(const Call &c, cudaStream_t st);
cudaError_t few_backward(const Call &c, cudaStream_t st);
cudaError_t forward(const Call &c, cudaStream_t st);
cudaError_t backward(const Call &c, cudaStream_t st);

}  // namespace xent
}  // namespace gdn
