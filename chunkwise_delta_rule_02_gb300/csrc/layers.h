// Launchers of the layer operators, called by layers_api.cu with checked arguments.
#pragma once

#include "layers.cuh"

namespace gdn {
namespace lay {

struct ConvCall {
    const dn_conv_shape *s;
    int N;                          // sequences
    const int32_t *cu;              // checked offsets in the workspace (packed), else null
    const dn_view *x, *y, *dy, *dx;
    const float *w, *bias;
    const void *s0, *dsT;
    void *sT, *ds0;
    float *dw, *dbias;
    float *part;                    // backward: partial sums
};

// rows of partial sums the backward writes
long long conv_part_rows(const dn_conv_shape *s);
cudaError_t conv_fwd(const ConvCall &c, cudaStream_t st);
cudaError_t conv_bwd(const ConvCall &c, cudaStream_t st);
cudaError_t conv_step(const ConvCall &c, cudaStream_t st);

struct NormCall {
    const dn_norm_shape *s;
    const dn_view *x, *z, *residual, *sum, *y, *dy, *dsum, *dx, *dz, *dresidual;
    const float *w, *res_scale;
    float *dw, *dres_scale, *part;
};
long long norm_part_rows(const dn_norm_shape *s);
cudaError_t norm_fwd(const NormCall &c, cudaStream_t st);
cudaError_t norm_bwd(const NormCall &c, cudaStream_t st);

}  // namespace lay
}  // namespace gdn
