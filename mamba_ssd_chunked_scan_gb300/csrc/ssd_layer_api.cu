// C ABI of the operators around the scan (residual norm, gated recurrence):
// argument checks and dispatch.  Nothing here allocates device memory; every launch is asynchronous
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

// A (rows, width) matrix of `es`-byte elements with `stride` elements between rows.
struct Mat {
    const void* p;
    int64_t rows, width, stride;
    size_t es;
    size_t span() const { return p && rows ? ((size_t)(rows - 1) * stride + width) * es : 0; }
};
// Whether two matrices share an element.  Column ranges of one wider matrix lie
// inside each other's span without touching.
bool touch(const Mat& a, const Mat& b) {
    if (!overlap(a.p, a.span(), b.p, b.span())) return false;
    if (a.stride == b.stride && a.es == b.es) {
        const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
        const size_t pitch = (size_t)a.stride * a.es;
        const Mat& lo = x < y ? a : b;
        const Mat& hi = x < y ? b : a;
        const size_t off = (x < y ? y - x : x - y) % pitch;
        return !(off >= (size_t)lo.width * lo.es && off + (size_t)hi.width * hi.es <= pitch);
    }
    return true;
}

int check_scan(const ssd_gate_scan_params_t* p) {
    if (!p) return SSD_ERR_INVALID_ARG;
    if (p->batch < 1 || p->seqlen < 1 || p->width < 1 || p->ndocs < 0) return SSD_ERR_INVALID_ARG;
    if (p->dtype != SSD_F32 && p->dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
    if (p->g_stride < p->width || p->x_stride < p->width) return SSD_ERR_INVALID_ARG;
    if (p->ndocs > 0 && p->batch != 1) return SSD_ERR_INVALID_ARG;
    const int64_t big = (int64_t)1 << 31;
    // token offsets and tile numbers are 32-bit; element offsets are 64-bit
    if (p->seqlen >= big - kScanTok || p->batch >= big || p->batch * p->seqlen >= big << 8 || p->g_stride >= big || p->x_stride >= big)
        return SSD_ERR_UNSUPPORTED;
    const int64_t tiles = ((p->seqlen + kScanTok - 1) / kScanTok) * ((p->width + kScanCh - 1) / kScanCh);
    if (tiles >= big / p->batch) return SSD_ERR_UNSUPPORTED;
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

size_t ssd_gate_scan_workspace_size(const ssd_gate_scan_params_t* p) {
    if (check_scan(p) != SSD_OK) return 0;
    return gate_scan_layout(p->batch, p->seqlen, p->width).total;
}

int ssd_gate_scan(const ssd_gate_scan_params_t* p, const void* g, const void* x, const float* initial_states,
                  const int32_t* cu_seqlens, void* y, float* final_states, void* workspace, size_t workspace_bytes,
                  void* stream) {
    const int rc = check_scan(p);
    if (rc != SSD_OK) return rc;
    if (!g || !x || !y || (p->ndocs > 0) != (cu_seqlens != nullptr)) return SSD_ERR_INVALID_ARG;
    const size_t es = elem(p->dtype);
    if (!aligned(g, es) || !aligned(x, es) || !aligned(y, es) || !aligned(initial_states, 4) ||
        !aligned(final_states, 4) || !aligned(cu_seqlens, 4))
        return SSD_ERR_INVALID_ARG;
    const size_t need = gate_scan_layout(p->batch, p->seqlen, p->width).total;
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return SSD_ERR_WORKSPACE;
    const int64_t rows = p->batch * p->seqlen, nst = p->ndocs > 0 ? p->ndocs : p->batch;
    const Mat in[] = {{g, rows, p->width, p->g_stride, es}, {x, rows, p->width, p->x_stride, es},
                      {initial_states, nst, p->width, p->width, 4}, {cu_seqlens, 1, p->ndocs + 1, p->ndocs + 1, 4}};
    const Mat out[] = {{y, rows, p->width, p->width, es}, {final_states, nst, p->width, p->width, 4},
                       {workspace, 1, (int64_t)need, (int64_t)need, 1}};
    for (int i = 0; i < 3; ++i) {
        for (const Mat& m : in)
            if (touch(out[i], m)) return SSD_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (touch(out[i], out[j])) return SSD_ERR_INVALID_ARG;
    }
    GateScanArgs a = {};
    a.batch = p->batch; a.seqlen = p->seqlen; a.width = p->width; a.dtype = p->dtype; a.ndocs = p->ndocs;
    a.g_stride = p->g_stride; a.x_stride = p->x_stride;
    a.g = g; a.x = x; a.init = initial_states; a.cu = cu_seqlens; a.y = y; a.fin = final_states;
    return launch_gate_scan(a, workspace, false, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

int ssd_gate_scan_bwd(const ssd_gate_scan_params_t* p, const void* g, const void* x, const void* y,
                      const float* initial_states, const int32_t* cu_seqlens, const void* dy,
                      const float* dfinal_states, void* dg, void* dx, float* dinitial_states, void* workspace,
                      size_t workspace_bytes, void* stream) {
    const int rc = check_scan(p);
    if (rc != SSD_OK) return rc;
    if (!g || !x || !y || !dy || !dg || !dx || (p->ndocs > 0) != (cu_seqlens != nullptr)) return SSD_ERR_INVALID_ARG;
    const size_t es = elem(p->dtype);
    if (!aligned(g, es) || !aligned(x, es) || !aligned(y, es) || !aligned(dy, es) || !aligned(dg, es) ||
        !aligned(dx, es) || !aligned(initial_states, 4) || !aligned(dfinal_states, 4) || !aligned(dinitial_states, 4) ||
        !aligned(cu_seqlens, 4))
        return SSD_ERR_INVALID_ARG;
    const size_t need = gate_scan_layout(p->batch, p->seqlen, p->width).total;
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return SSD_ERR_WORKSPACE;
    const int64_t rows = p->batch * p->seqlen, nst = p->ndocs > 0 ? p->ndocs : p->batch;
    const int64_t w = p->width;
    const Mat in[] = {{g, rows, w, p->g_stride, es}, {x, rows, w, p->x_stride, es}, {y, rows, w, w, es}, {dy, rows, w, w, es},
                      {initial_states, nst, w, w, 4}, {dfinal_states, nst, w, w, 4},
                      {cu_seqlens, 1, p->ndocs + 1, p->ndocs + 1, 4}};
    const Mat out[] = {{dg, rows, w, p->g_stride, es}, {dx, rows, w, p->x_stride, es}, {dinitial_states, nst, w, w, 4},
                       {workspace, 1, (int64_t)need, (int64_t)need, 1}};
    for (int i = 0; i < 4; ++i) {
        for (const Mat& m : in)
            if (touch(out[i], m)) return SSD_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (touch(out[i], out[j])) return SSD_ERR_INVALID_ARG;
    }
    GateScanArgs a = {};
    a.batch = p->batch; a.seqlen = p->seqlen; a.width = p->width; a.dtype = p->dtype; a.ndocs = p->ndocs;
    a.g_stride = p->g_stride; a.x_stride = p->x_stride;
    a.g = g; a.x = x; a.init = initial_states; a.cu = cu_seqlens; a.y = const_cast<void*>(y);
    a.dy = dy; a.dfin = dfinal_states; a.dg = dg; a.dx = dx; a.dinit = dinitial_states;
    return launch_gate_scan(a, workspace, true, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

int ssd_gate_scan_step(int64_t batch, int32_t width, int32_t dtype, int64_t g_stride, int64_t x_stride, const void* g,
                       const void* x, const float* state_in, float* state_out, void* y, void* stream) {
    if (batch < 0 || width < 1 || g_stride < width || x_stride < width) return SSD_ERR_INVALID_ARG;
    if (dtype != SSD_F32 && dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
    if (batch == 0) return SSD_OK;
    if (batch >= ((int64_t)1 << 36) / width || g_stride >= (int64_t)1 << 31 || x_stride >= (int64_t)1 << 31) return SSD_ERR_UNSUPPORTED;
    if (!g || !x || !state_in || !state_out || !y) return SSD_ERR_INVALID_ARG;
    const size_t es = elem(dtype);
    if (!aligned(g, es) || !aligned(x, es) || !aligned(y, es) || !aligned(state_in, 4) || !aligned(state_out, 4))
        return SSD_ERR_INVALID_ARG;
    const Mat mg = {g, batch, width, g_stride, es}, mx = {x, batch, width, x_stride, es}, my = {y, batch, width, width, es};
    const Mat si = {state_in, batch, width, width, 4}, so = {state_out, batch, width, width, 4};
    if (touch(my, mg) || touch(my, mx) || touch(my, si) || touch(my, so) || touch(so, mg) || touch(so, mx) ||
        (state_in != state_out && touch(so, si)))
        return SSD_ERR_INVALID_ARG;
    GateStepArgs a;
    a.batch = batch; a.width = width; a.dtype = dtype; a.g_stride = g_stride; a.x_stride = x_stride;
    a.g = g; a.x = x; a.state_in = state_in; a.state_out = state_out; a.y = y;
    return launch_gate_scan_step(a, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
