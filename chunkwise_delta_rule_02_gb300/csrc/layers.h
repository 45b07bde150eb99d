// Launchers of the layer operators, called by layers_api.cu with checked arguments.
#pragma once

#include <cuda.h>

#include "layers.cuh"

namespace gdn {
namespace lay {

// Whether tensor maps can be made at all (the driver has the entry point).
bool has_tensor_maps();
// Tensor map of a [planes][rows][cols] array of bf16 or float32, boxes of `wide` columns x `high` rows; pitches in elements.
// `swizzle`: 0, 64 or
// 128 bytes.  Zero is read outside.  False where the array does not meet a map's rules.
bool tensor_map(CUtensorMap *m, bool f32, const void *p, long long cols, long long rows, long long planes, long long row_pitch,
                long long plane_pitch, int wide, int high, int swizzle);

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

struct DropCall {
    const dn_dropout_shape *s;
    const dn_view *x, *residual, *y;
    const int64_t *rng;
};
cudaError_t dropout(const DropCall &c, cudaStream_t st);

}  // namespace lay
}  // namespace gdn
