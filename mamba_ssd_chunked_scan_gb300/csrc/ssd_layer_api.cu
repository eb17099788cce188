// C ABI of the operators around the scan (residual norm): argument checks and
// dispatch.  Nothing here allocates device memory; every launch is asynchronous
// on the caller's stream.
#include "ssd_common.cuh"
#include "ssd_kernels.h"

using namespace ssd;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool known(int dtype) { return dtype == SSD_F32 || dtype == SSD_BF16 || dtype == SSD_E4M3; }
size_t elem(int dtype) { return dtype == SSD_F32 ? 4 : dtype == SSD_BF16 ? 2 : 1; }

// Whether [a, a + na) and [b, b + nb) share a byte (NULL shares none).
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + nb && y < x + na;
}
// Overlap other than being the same array with elements of the same size.
bool clash(const void* a, size_t na, const void* b, size_t nb) { return overlap(a, na, b, nb) && !(a == b && na == nb); }

// Types and width of the residual norm; SSD_OK or the status to return.
int check_norm(int64_t rows, int32_t width, int32_t dtype, int32_t residual_dtype) {
    if (rows < 0 || width < 1) return SSD_ERR_INVALID_ARG;
    if (dtype != SSD_F32 && dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
    if (residual_dtype != SSD_F32 && !(residual_dtype == SSD_BF16 && dtype == SSD_BF16)) return SSD_ERR_INVALID_ARG;
    if (width > kAddNormMaxWidth || rows >= ((int64_t)1 << 31)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

}  // namespace

extern "C" {

int ssd_add_norm(int64_t rows, int32_t width, int32_t dtype, int32_t residual_dtype, int32_t out_dtype,
                 const void* x, const void* residual, const float* weight, float eps, void* out, float* scales,
                 void* residual_out, float* rstd, void* stream) {
    if (!known(out_dtype)) return SSD_ERR_INVALID_ARG;
    const int rc = check_norm(rows, width, dtype, residual_dtype);
    if (rc != SSD_OK) return rc;
    if (out_dtype != dtype && out_dtype != SSD_E4M3) return SSD_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || eps > 3.0e38f) return SSD_ERR_INVALID_ARG;   // rejects NaN and inf
    if (rows == 0) return SSD_OK;
    if (!x || !weight || !out || (out_dtype == SSD_E4M3 && !scales)) return SSD_ERR_INVALID_ARG;
    if (!aligned(x, elem(dtype)) || !aligned(out, elem(out_dtype)) || !aligned(residual, elem(residual_dtype)) ||
        !aligned(residual_out, elem(residual_dtype)) || !aligned(weight, 4) || !aligned(scales, 4) || !aligned(rstd, 4))
        return SSD_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * width, nx = n * elem(dtype), no = n * elem(out_dtype), nr = n * elem(residual_dtype);
    const size_t nw = (size_t)width * 4, ns = (size_t)rows * 4;
    if (out_dtype != SSD_E4M3) scales = nullptr;
    if (clash(out, no, x, nx) || clash(out, no, residual, nr) || clash(residual_out, nr, residual, nr) ||
        clash(residual_out, nr, x, nx) || overlap(residual_out, nr, out, no) || overlap(out, no, weight, nw) ||
        overlap(residual_out, nr, weight, nw))
        return SSD_ERR_INVALID_ARG;
    float* const small[2] = {scales, rstd};
    for (float* s : small)
        if (overlap(s, ns, x, nx) || overlap(s, ns, residual, nr) || overlap(s, ns, weight, nw) ||
            overlap(s, ns, out, no) || overlap(s, ns, residual_out, nr))
            return SSD_ERR_INVALID_ARG;
    if (overlap(scales, ns, rstd, ns)) return SSD_ERR_INVALID_ARG;
    AddNormArgs a;
    a.rows = rows; a.width = width; a.dtype = dtype; a.residual_dtype = residual_dtype; a.out_dtype = out_dtype;
    a.eps = eps; a.x = x; a.residual = residual; a.weight = weight; a.out = out; a.scales = scales;
    a.residual_out = residual_out; a.rstd = rstd;
    return launch_add_norm(a, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

size_t ssd_add_norm_bwd_workspace_size(int64_t rows, int32_t width) {
    if (rows < 1 || check_norm(rows, width, SSD_F32, SSD_F32) != SSD_OK) return 0;
    return (size_t)add_norm_bwd_shares(rows, width) * width * sizeof(float);
}

int ssd_add_norm_bwd(int64_t rows, int32_t width, int32_t dtype, int32_t residual_dtype, const void* dout,
                     const void* h, const float* weight, const float* rstd, const void* dresidual_out, void* dx,
                     void* dresidual, float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_norm(rows, width, dtype, residual_dtype);
    if (rc != SSD_OK) return rc;
    if (!dweight || !aligned(dweight, 4)) return SSD_ERR_INVALID_ARG;
    if (rows == 0)
        return cudaMemsetAsync(dweight, 0, (size_t)width * 4, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    if (!dout || !h || !weight || !rstd || (!dx && !dresidual)) return SSD_ERR_INVALID_ARG;
    const size_t et = elem(dtype), er = elem(residual_dtype);
    if (!aligned(dout, et) || !aligned(dx, et) || !aligned(h, er) || !aligned(dresidual_out, er) ||
        !aligned(dresidual, er) || !aligned(weight, 4) || !aligned(rstd, 4))
        return SSD_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * width, nt = n * et, nr = n * er, nw = (size_t)width * 4, ns = (size_t)rows * 4;
    const size_t need = ssd_add_norm_bwd_workspace_size(rows, width);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return SSD_ERR_WORKSPACE;
    // dx and dresidual may each replace an incoming gradient of their own type
    if (clash(dx, nt, dout, nt) || overlap(dx, nt, h, nr) || clash(dx, nt, dresidual_out, nr) ||
        clash(dresidual, nr, dout, nt) || overlap(dresidual, nr, h, nr) || clash(dresidual, nr, dresidual_out, nr) ||
        overlap(dx, nt, dresidual, nr))
        return SSD_ERR_INVALID_ARG;
    struct { const void* p; size_t n; } const in[] = {{dout, nt}, {h, nr}, {dresidual_out, nr}, {weight, nw},
                                                      {rstd, ns}, {dx, nt}, {dresidual, nr}};
    for (const auto& b : in)
        if (overlap(dweight, nw, b.p, b.n) || overlap(workspace, need, b.p, b.n)) return SSD_ERR_INVALID_ARG;
    if (overlap(dx, nt, weight, nw) || overlap(dresidual, nr, weight, nw) || overlap(dx, nt, rstd, ns) ||
        overlap(dresidual, nr, rstd, ns) || overlap(dweight, nw, workspace, need))
        return SSD_ERR_INVALID_ARG;
    AddNormBwdArgs a;
    a.rows = rows; a.width = width; a.dtype = dtype; a.residual_dtype = residual_dtype;
    a.dout = dout; a.h = h; a.weight = weight; a.rstd = rstd; a.dres = dresidual_out;
    a.dx = dx; a.dres_out = dresidual; a.dweight = dweight; a.shares = (float*)workspace;
    return launch_add_norm_bwd(a, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
