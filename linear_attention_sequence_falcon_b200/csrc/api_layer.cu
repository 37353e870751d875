// api_layer.cu -- the C ABI of the layer operators (declared in
// include/falcon.h): argument validation, empty sizes, dispatch to the
// kernels of k_scan.cu and k_norm.cu.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/falcon.h"
#include "kernels.h"
#include "params_layer.h"

using namespace falcon;

static_assert(kScanBlock == FALCON_SCAN_BLOCK && kNormMaxD == FALCON_NORM_MAX_D, "the header's constants");

namespace {

bool dtype_ok(int t) { return t == FALCON_F32 || t == FALCON_BF16; }

int done(int rc) {
    if (rc != 0) return rc;
    return cudaGetLastError() == cudaSuccess ? FALCON_OK : FALCON_ERR_LAUNCH;
}

// a row stride of `rows` rows of `len` elements: at least the row, and small
// enough that an element offset fits 63 bits
bool stride_ok(long long ld, long long rows, long long len) {
    if (rows <= 1) return true;
    return ld >= len && ld <= (1ll << 60) / rows;
}

bool ws_ok(const void *ws, size_t bytes, size_t need) {
    return need == 0 || (ws && bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0);
}

// dst = src, or zeros without src
int fill_f32(float *dst, const float *src, size_t n, cudaStream_t s) {
    if (!dst || n == 0 || dst == src) return FALCON_OK;
    const cudaError_t e = src ? cudaMemcpyAsync(dst, src, n * sizeof(float), cudaMemcpyDeviceToDevice, s)
                              : cudaMemsetAsync(dst, 0, n * sizeof(float), s);
    if (e == cudaSuccess) return FALCON_OK;
    cudaGetLastError();
    return FALCON_ERR_LAUNCH;
}

// The limit of a grid's one axis; token counts stay far enough under it that
// a tile's tokens behind the end still have int positions.
constexpr long long kMaxItems = 0x7fffffffll;

bool scan_sizes_ok(int N, int L, int D) {
    if (N < 0 || L < 0 || L > (1 << 30) || D < 0) return false;
    const long long items = (long long)N * ((D + 31) / 32);
    return items <= kMaxItems / 32;
}

// a row stride of the recurrence: the kernels place a tile's elements (at most
// 512 tokens) by 32-bit byte offsets
constexpr long long kScanMaxStride = 1 << 21;
bool scan_stride_ok(long long ld, long long rows, long long D) {
    return D <= kScanMaxStride && stride_ok(ld, rows, D) && (rows <= 1 || ld <= kScanMaxStride);
}

size_t marks_floats(int N, int L, int D) { return (size_t)N * ((L + kScanBlock - 1) / kScanBlock) * D; }

}  // namespace

extern "C" int falcon_scan(falcon_dtype dtype, const void *x, const void *f, const unsigned char *reset,
                           const float *initial_state, int N, int L, int D, long long x_stride, long long f_stride,
                           void *out, float *final_state, float *marks, cudaStream_t stream) {
    if (!dtype_ok(dtype)) return FALCON_ERR_ENUM;
    const long long rows = (long long)N * L;
    if (!scan_sizes_ok(N, L, D) || !scan_stride_ok(x_stride, rows, D) || !scan_stride_ok(f_stride, rows, D))
        return FALCON_ERR_SHAPE;
    if (N == 0 || D == 0) return FALCON_OK;
    if (L == 0) return fill_f32(final_state, initial_state, (size_t)N * D, stream);
    if (!x || !f || !out) return FALCON_ERR_NULL;
    ScanParams p{};
    p.N = N; p.L = L; p.D = D; p.ldx = rows > 1 ? x_stride : D; p.ldf = rows > 1 ? f_stride : D;
    p.x = x; p.f = f; p.reset = reset; p.init_state = initial_state;
    p.out = out; p.final_state = final_state; p.marks = marks;
    return done(dtype == FALCON_BF16 ? launch_scan<__nv_bfloat16>(p, stream) : launch_scan<float>(p, stream));
}

extern "C" int falcon_scan_bwd_workspace_size(falcon_dtype dtype, int N, int L, int D, int has_marks,
                                              size_t *bytes) {
    if (!bytes) return FALCON_ERR_NULL;
    *bytes = 0;
    if (!dtype_ok(dtype)) return FALCON_ERR_ENUM;
    if (!scan_sizes_ok(N, L, D)) return FALCON_ERR_SHAPE;
    if (!has_marks) *bytes = marks_floats(N, L, D) * sizeof(float);
    return FALCON_OK;
}

extern "C" int falcon_scan_bwd_ws(falcon_dtype dtype, const void *x, const void *f, const unsigned char *reset,
                                  const float *initial_state, const float *marks, int N, int L, int D,
                                  long long x_stride, long long f_stride, const void *dout, const float *dstate,
                                  void *dx, long long dx_stride, void *df, long long df_stride, float *dinitial,
                                  void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!dtype_ok(dtype)) return FALCON_ERR_ENUM;
    const long long rows = (long long)N * L;
    if (!scan_sizes_ok(N, L, D) || !scan_stride_ok(x_stride, rows, D) || !scan_stride_ok(f_stride, rows, D) ||
        !scan_stride_ok(dx_stride, rows, D) || !scan_stride_ok(df_stride, rows, D))
        return FALCON_ERR_SHAPE;
    if (N == 0 || D == 0) return FALCON_OK;
    if (L == 0) return fill_f32(dinitial, dstate, (size_t)N * D, stream);
    if (!x || !f || !dout || !dx || !df) return FALCON_ERR_NULL;
    const bool bf16 = dtype == FALCON_BF16;
    if (!marks) {
        if (!ws_ok(workspace, workspace_bytes, marks_floats(N, L, D) * sizeof(float))) return FALCON_ERR_WORKSPACE;
        ScanParams q{};
        q.N = N; q.L = L; q.D = D; q.ldx = rows > 1 ? x_stride : D; q.ldf = rows > 1 ? f_stride : D;
        q.x = x; q.f = f; q.reset = reset; q.init_state = initial_state;
        q.marks = static_cast<float *>(workspace);
        const int rc = done(bf16 ? launch_scan<__nv_bfloat16>(q, stream) : launch_scan<float>(q, stream));
        if (rc) return rc;
        marks = q.marks;
    }
    ScanBwdParams p{};
    p.N = N; p.L = L; p.D = D;
    const bool one = rows <= 1;  // no second row: the strides say nothing
    p.ldx = one ? D : x_stride; p.ldf = one ? D : f_stride; p.lddx = one ? D : dx_stride; p.lddf = one ? D : df_stride;
    p.x = x; p.f = f; p.reset = reset; p.marks = marks; p.dout = dout; p.dstate = dstate;
    p.dx = dx; p.df = df; p.dinitial = dinitial;
    return done(bf16 ? launch_scan_bwd<__nv_bfloat16>(p, stream) : launch_scan_bwd<float>(p, stream));
}

extern "C" int falcon_scan_step(falcon_dtype dtype, const void *x, const void *f, const float *state, int N, int D,
                                long long x_stride, long long f_stride, float *state_out, void *out,
                                cudaStream_t stream) {
    if (!dtype_ok(dtype)) return FALCON_ERR_ENUM;
    if (!scan_sizes_ok(N, 1, D) || !stride_ok(x_stride, N, D) || !stride_ok(f_stride, N, D)) return FALCON_ERR_SHAPE;
    if (N == 0 || D == 0) return FALCON_OK;
    if (!x || !f || !state || !state_out || !out) return FALCON_ERR_NULL;
    ScanStepParams p{};
    p.N = N; p.D = D; p.ldx = x_stride; p.ldf = f_stride;
    p.x = x; p.f = f; p.state = state; p.state_out = state_out; p.out = out;
    return done(dtype == FALCON_BF16 ? launch_scan_step<__nv_bfloat16>(p, stream)
                                     : launch_scan_step<float>(p, stream));
}

namespace {

// the sizes, eps and strides that both passes of the gated norm share
int gate_check(int dtype, long long o_sb, long long o_sh, long long o_sl, const void *gate, long long gate_stride,
               float eps, int B, int H, int L, int d) {
    if (!dtype_ok(dtype)) return FALCON_ERR_ENUM;
    if (B < 0 || H < 0 || L < 0 || d < 1 || d > kNormMaxD) return FALCON_ERR_SHAPE;
    const long long tokens = (long long)B * L;
    if (tokens > kMaxItems || tokens * H > (1ll << 46) || (long long)H * d > kMaxItems) return FALCON_ERR_SHAPE;
    const long long far = 1ll << 60;
    if (o_sb < 0 || o_sh < 0 || o_sl < 0 || (B > 1 && o_sb > far / B) || (H > 1 && o_sh > far / H) ||
        (L > 1 && o_sl > far / L))
        return FALCON_ERR_SHAPE;
    if (gate && !stride_ok(gate_stride, tokens, (long long)H * d)) return FALCON_ERR_SHAPE;
    if (!(eps >= 0.f)) return FALCON_ERR_UNSUPPORTED;
    return FALCON_OK;
}

int residual_check(int dtype, float eps, int R, int D) {
    if (!dtype_ok(dtype)) return FALCON_ERR_ENUM;
    if (R < 0 || D < 1 || D > kNormMaxD) return FALCON_ERR_SHAPE;
    if (!(eps >= 0.f)) return FALCON_ERR_UNSUPPORTED;
    return FALCON_OK;
}

}  // namespace

extern "C" int falcon_norm_gate(falcon_dtype dtype, const void *o, long long o_sb, long long o_sh, long long o_sl,
                                const void *gate, long long gate_stride, const float *weight, int per_head,
                                float eps, int B, int H, int L, int d, void *out, cudaStream_t stream) {
    const int rc = gate_check(dtype, o_sb, o_sh, o_sl, gate, gate_stride, eps, B, H, L, d);
    if (rc) return rc;
    if ((long long)B * H * L == 0) return FALCON_OK;
    if (!o || !out) return FALCON_ERR_NULL;
    NormGateParams p{};
    p.B = B; p.H = H; p.L = L; p.d = d; p.per_head = per_head != 0;
    p.o_sb = o_sb; p.o_sh = o_sh; p.o_sl = o_sl; p.ldg = gate_stride; p.eps = eps;
    p.o = o; p.gate = gate; p.weight = weight; p.out = out;
    return done(dtype == FALCON_BF16 ? launch_norm_gate<__nv_bfloat16>(p, stream)
                                     : launch_norm_gate<float>(p, stream));
}

extern "C" int falcon_norm_gate_bwd_workspace_size(falcon_dtype dtype, int B, int H, int L, int d, size_t *bytes) {
    if (!bytes) return FALCON_ERR_NULL;
    *bytes = 0;
    const int rc = gate_check(dtype, 0, 0, 0, nullptr, 0, 0.f, B, H, L, d);
    if (rc) return rc;
    if ((long long)B * H * L != 0) *bytes = norm_gate_bwd_ws_bytes(dtype == FALCON_BF16, B, H, L, d);
    return FALCON_OK;
}

extern "C" int falcon_norm_gate_bwd_ws(falcon_dtype dtype, const void *o, long long o_sb, long long o_sh,
                                       long long o_sl, const void *gate, long long gate_stride, const float *weight,
                                       int per_head, float eps, int B, int H, int L, int d, const void *dout,
                                       void *d_o, long long d_o_sb, long long d_o_sh, long long d_o_sl, void *dgate,
                                       long long dgate_stride, float *dweight, void *workspace,
                                       size_t workspace_bytes, cudaStream_t stream) {
    int rc = gate_check(dtype, o_sb, o_sh, o_sl, gate, gate_stride, eps, B, H, L, d);
    if (!rc) rc = gate_check(dtype, d_o_sb, d_o_sh, d_o_sl, dgate, dgate_stride, eps, B, H, L, d);
    if (rc) return rc;
    if ((long long)B * H * L == 0)
        return fill_f32(dweight, nullptr, (size_t)d * (per_head ? H : 1), stream);
    if (!o || !dout || !d_o || (gate == nullptr) != (dgate == nullptr)) return FALCON_ERR_NULL;
    if (!ws_ok(workspace, workspace_bytes, norm_gate_bwd_ws_bytes(dtype == FALCON_BF16, B, H, L, d)))
        return FALCON_ERR_WORKSPACE;
    NormGateParams p{};
    p.B = B; p.H = H; p.L = L; p.d = d; p.per_head = per_head != 0;
    p.o_sb = o_sb; p.o_sh = o_sh; p.o_sl = o_sl; p.ldg = gate_stride; p.eps = eps;
    p.o = o; p.gate = gate; p.weight = weight; p.dout = dout;
    p.d_o = d_o; p.do_sb = d_o_sb; p.do_sh = d_o_sh; p.do_sl = d_o_sl;
    p.dgate = dgate; p.lddg = dgate_stride; p.dweight = dweight; p.ws = static_cast<float *>(workspace);
    return done(dtype == FALCON_BF16 ? launch_norm_gate_bwd<__nv_bfloat16>(p, stream)
                                     : launch_norm_gate_bwd<float>(p, stream));
}

extern "C" int falcon_residual_norm(falcon_dtype dtype, const void *r, const void *y, const float *scale,
                                    const float *weight, float eps, int R, int D, void *r_out, void *h,
                                    cudaStream_t stream) {
    const int rc = residual_check(dtype, eps, R, D);
    if (rc) return rc;
    if (R == 0) return FALCON_OK;
    if (!r || !h) return FALCON_ERR_NULL;
    ResidualNormParams p{};
    p.R = R; p.D = D; p.eps = eps; p.r = r; p.y = y; p.scale = scale; p.weight = weight; p.r_out = r_out; p.h = h;
    return done(dtype == FALCON_BF16 ? launch_residual_norm<__nv_bfloat16>(p, stream)
                                     : launch_residual_norm<float>(p, stream));
}

extern "C" int falcon_residual_norm_bwd_workspace_size(falcon_dtype dtype, int R, int D, size_t *bytes) {
    if (!bytes) return FALCON_ERR_NULL;
    *bytes = 0;
    const int rc = residual_check(dtype, 0.f, R, D);
    if (rc) return rc;
    if (R != 0) *bytes = residual_norm_bwd_ws_bytes(dtype == FALCON_BF16, R, D);
    return FALCON_OK;
}

extern "C" int falcon_residual_norm_bwd_ws(falcon_dtype dtype, const void *r_out, const void *y, const float *scale,
                                           const float *weight, const void *dh, const void *dr_out, float eps, int R,
                                           int D, void *dr, void *dy, float *dscale, float *dweight,
                                           void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    const int rc = residual_check(dtype, eps, R, D);
    if (rc) return rc;
    if (R == 0) {
        const int e = fill_f32(dscale, nullptr, D, stream);
        return e ? e : fill_f32(dweight, nullptr, D, stream);
    }
    if (!r_out || !dh || !dr || (dscale && !y)) return FALCON_ERR_NULL;
    if (!ws_ok(workspace, workspace_bytes, residual_norm_bwd_ws_bytes(dtype == FALCON_BF16, R, D)))
        return FALCON_ERR_WORKSPACE;
    ResidualNormParams p{};
    p.R = R; p.D = D; p.eps = eps; p.r = r_out; p.y = y; p.scale = scale; p.weight = weight;
    p.dh = dh; p.dr_out = dr_out; p.dr = dr; p.dy = dy; p.dscale = dscale; p.dweight = dweight;
    p.ws = static_cast<float *>(workspace);
    return done(dtype == FALCON_BF16 ? launch_residual_norm_bwd<__nv_bfloat16>(p, stream)
                                     : launch_residual_norm_bwd<float>(p, stream));
}
