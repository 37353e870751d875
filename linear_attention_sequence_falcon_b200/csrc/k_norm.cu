// k_norm.cu -- the norms around a block: falcon_norm_gate (behind it, with
// its gate) and falcon_residual_norm (in front of it, with the residual add),
// forward and backward.
//
// One warp per row; the weights' gradients come from partial sums over runs
// of rows, one thread per channel, and a second kernel that adds the partial
// sums in order.
#include "common.cuh"
#include "kernels.h"
#include "params_layer.h"

namespace falcon {

namespace {

constexpr int kRuns = 128;  // partial sums per channel

// 1/sqrt(ms + eps); a row of zeros with eps = 0 is left as zeros
__device__ __forceinline__ float inv_rms(float ms, float eps) {
    const float v = ms + eps;
    return v == 0.f ? 0.f : rsqrtf(v);
}

struct GateRow {
    long long o, g, out, d_o, dg;  // element offsets of the row's first channel
    int h;
};

__device__ __forceinline__ GateRow gate_row(const NormGateParams &p, long long row) {
    // rows in the order of the output: (b, l, h)
    const long long token = row / p.H;
    GateRow r;
    r.h = (int)(row % p.H);
    const int b = (int)(token / p.L), l = (int)(token % p.L);
    r.o = b * p.o_sb + r.h * p.o_sh + l * p.o_sl;
    r.d_o = b * p.do_sb + r.h * p.do_sh + l * p.do_sl;
    r.out = row * p.d;
    r.g = token * p.ldg + (long long)r.h * p.d;
    r.dg = token * p.lddg + (long long)r.h * p.d;
    return r;
}

__device__ __forceinline__ float sigmoid(float z) {
    const float e = expf(-fabsf(z)), big = 1.f / (1.f + e);
    return z < 0.f ? e * big : big;
}

template <typename T>
__global__ void __launch_bounds__(128) norm_gate_kernel(NormGateParams p) {
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= (long long)p.B * p.L * p.H) return;
    const GateRow r = gate_row(p, row);
    const T *o = static_cast<const T *>(p.o) + r.o;
    float ss = 0.f;
    for (int c = lane; c < p.d; c += 32) ss += to_f32(o[c]) * to_f32(o[c]);
    const float rstd = inv_rms(group_sum<32>(ss) / p.d, p.eps);
    const float *w = p.weight ? p.weight + (p.per_head ? (long long)r.h * p.d : 0) : nullptr;
    for (int c = lane; c < p.d; c += 32) {
        float y = to_f32(o[c]) * rstd * (w ? w[c] : 1.f);
        if (p.gate) {
            const float z = to_f32(static_cast<const T *>(p.gate)[r.g + c]);
            y *= z * sigmoid(z);
        }
        static_cast<T *>(p.out)[r.out + c] = from_f32<T>(y);
    }
}

// ws: rstd of every row, then the partial sums
template <typename T>
__global__ void __launch_bounds__(128) norm_gate_bwd_kernel(NormGateParams p) {
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= (long long)p.B * p.L * p.H) return;
    const GateRow r = gate_row(p, row);
    const T *o = static_cast<const T *>(p.o) + r.o;
    const T *dout = static_cast<const T *>(p.dout) + r.out;
    const float *w = p.weight ? p.weight + (p.per_head ? (long long)r.h * p.d : 0) : nullptr;
    float ss = 0.f, dot = 0.f;
    for (int c = lane; c < p.d; c += 32) {
        const float ov = to_f32(o[c]);
        float e = to_f32(dout[c]) * (w ? w[c] : 1.f);
        if (p.gate) {
            const float z = to_f32(static_cast<const T *>(p.gate)[r.g + c]);
            e *= z * sigmoid(z);
        }
        ss += ov * ov;
        dot += e * ov;
    }
    const float rstd = inv_rms(group_sum<32>(ss) / p.d, p.eps);
    const float m = group_sum<32>(dot) * rstd / p.d;
    if (lane == 0) p.ws[row] = rstd;
    for (int c = lane; c < p.d; c += 32) {
        const float n = to_f32(o[c]) * rstd, wc = w ? w[c] : 1.f, dy = to_f32(dout[c]);
        float act = 1.f;
        if (p.gate) {
            const float z = to_f32(static_cast<const T *>(p.gate)[r.g + c]), s = sigmoid(z);
            act = z * s;
            static_cast<T *>(p.dgate)[r.dg + c] = from_f32<T>(dy * n * wc * (s * (1.f + z * (1.f - s))));
        }
        static_cast<T *>(p.d_o)[r.d_o + c] = from_f32<T>(rstd * (dy * act * wc - n * m));
    }
}

// partial sums: block (run, head), one thread per channel
template <typename T>
__global__ void __launch_bounds__(256) norm_gate_dw_kernel(NormGateParams p) {
    const long long tokens = (long long)p.B * p.L;
    const long long t0 = tokens * blockIdx.x / kRuns, t1 = tokens * (blockIdx.x + 1) / kRuns;
    const int h = blockIdx.y;
    float *part = p.ws + tokens * p.H + ((long long)blockIdx.x * p.H + h) * p.d;
    for (int c = threadIdx.x; c < p.d; c += 256) {
        float acc = 0.f;
        for (long long t = t0; t < t1; ++t) {
            const GateRow r = gate_row(p, t * p.H + h);
            float e = to_f32(static_cast<const T *>(p.dout)[r.out + c]);
            if (p.gate) {
                const float z = to_f32(static_cast<const T *>(p.gate)[r.g + c]);
                e *= z * sigmoid(z);
            }
            acc = fmaf(e, to_f32(static_cast<const T *>(p.o)[r.o + c]) * p.ws[t * p.H + h], acc);
        }
        part[c] = acc;
    }
}

// out[c] = sum over i of part[i*n + c], in order
__global__ void __launch_bounds__(128) sum_parts_kernel(const float *part, int parts, long long n, float *out) {
    const long long c = (long long)blockIdx.x * 128 + threadIdx.x;
    if (c >= n) return;
    float acc = 0.f;
    for (int i = 0; i < parts; ++i) acc += part[i * n + c];
    out[c] = acc;
}

template <typename T>
__global__ void __launch_bounds__(128) residual_norm_kernel(ResidualNormParams p) {
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= p.R) return;
    const long long at = row * p.D;
    const T *r = static_cast<const T *>(p.r) + at;
    const T *y = p.y ? static_cast<const T *>(p.y) + at : nullptr;
    float ss = 0.f;
    for (int c = lane; c < p.D; c += 32) {
        float v = to_f32(r[c]);
        if (y) v = fmaf(p.scale ? p.scale[c] : 1.f, to_f32(y[c]), v);
        ss += v * v;
    }
    const float rstd = inv_rms(group_sum<32>(ss) / p.D, p.eps);
    for (int c = lane; c < p.D; c += 32) {
        float v = to_f32(r[c]);
        if (y) v = fmaf(p.scale ? p.scale[c] : 1.f, to_f32(y[c]), v);
        if (p.r_out) static_cast<T *>(p.r_out)[at + c] = from_f32<T>(v);
        static_cast<T *>(p.h)[at + c] = from_f32<T>(v * rstd * (p.weight ? p.weight[c] : 1.f));
    }
}

// ws: rstd and mean(e n) of every row, then the partial sums
template <typename T>
__global__ void __launch_bounds__(128) residual_norm_stats_kernel(ResidualNormParams p) {
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= p.R) return;
    const T *r = static_cast<const T *>(p.r) + row * p.D;
    const T *dh = static_cast<const T *>(p.dh) + row * p.D;
    float ss = 0.f, dot = 0.f;
    for (int c = lane; c < p.D; c += 32) {
        const float v = to_f32(r[c]);
        ss += v * v;
        dot += to_f32(dh[c]) * (p.weight ? p.weight[c] : 1.f) * v;
    }
    const float rstd = inv_rms(group_sum<32>(ss) / p.D, p.eps);
    const float m = group_sum<32>(dot) * rstd / p.D;
    if (lane == 0) { p.ws[2 * row] = rstd; p.ws[2 * row + 1] = m; }
}

// the rows' gradients and the partial sums: block (run, 256 channels)
template <typename T>
__global__ void __launch_bounds__(256) residual_norm_bwd_kernel(ResidualNormParams p) {
    const int c = blockIdx.y * 256 + threadIdx.x;
    if (c >= p.D) return;
    const long long r0 = (long long)p.R * blockIdx.x / kRuns, r1 = (long long)p.R * (blockIdx.x + 1) / kRuns;
    const float w = p.weight ? p.weight[c] : 1.f, sc = p.scale ? p.scale[c] : 1.f;
    float dw = 0.f, ds = 0.f;
    for (long long row = r0; row < r1; ++row) {
        const long long at = row * p.D + c;
        const float rstd = p.ws[2 * row], m = p.ws[2 * row + 1];
        const float n = to_f32(static_cast<const T *>(p.r)[at]) * rstd, dh = to_f32(static_cast<const T *>(p.dh)[at]);
        float t = rstd * (dh * w - n * m);
        if (p.dr_out) t += to_f32(static_cast<const T *>(p.dr_out)[at]);
        dw = fmaf(dh, n, dw);
        if (p.dscale) ds = fmaf(t, to_f32(static_cast<const T *>(p.y)[at]), ds);
        static_cast<T *>(p.dr)[at] = from_f32<T>(t);
        if (p.dy) static_cast<T *>(p.dy)[at] = from_f32<T>(t * sc);
    }
    float *part = p.ws + 2ll * p.R;
    part[(long long)blockIdx.x * p.D + c] = dw;
    part[((long long)kRuns + blockIdx.x) * p.D + c] = ds;
}

unsigned row_blocks(long long rows) { return (unsigned)((rows + 3) / 4); }

}  // namespace

size_t norm_gate_bwd_ws_bytes(int, int B, int H, int L, int d) {
    return sizeof(float) * ((size_t)B * H * L + (size_t)kRuns * H * d);
}
size_t residual_norm_bwd_ws_bytes(int, int R, int D) {
    return sizeof(float) * (2 * (size_t)R + 2 * (size_t)kRuns * D);
}

template <typename T> int launch_norm_gate(const NormGateParams &p, cudaStream_t s) {
    norm_gate_kernel<T><<<row_blocks((long long)p.B * p.L * p.H), 128, 0, s>>>(p);
    return 0;
}
template <typename T> int launch_norm_gate_bwd(const NormGateParams &p, cudaStream_t s) {
    const long long rows = (long long)p.B * p.L * p.H;
    norm_gate_bwd_kernel<T><<<row_blocks(rows), 128, 0, s>>>(p);
    if (!p.dweight) return 0;
    norm_gate_dw_kernel<T><<<dim3(kRuns, p.H), 256, 0, s>>>(p);
    const long long n = (long long)p.d * (p.per_head ? p.H : 1);
    sum_parts_kernel<<<(unsigned)((n + 127) / 128), 128, 0, s>>>(p.ws + rows, p.per_head ? kRuns : kRuns * p.H, n,
                                                                 p.dweight);
    return 0;
}
template <typename T> int launch_residual_norm(const ResidualNormParams &p, cudaStream_t s) {
    residual_norm_kernel<T><<<row_blocks(p.R), 128, 0, s>>>(p);
    return 0;
}
template <typename T> int launch_residual_norm_bwd(const ResidualNormParams &p, cudaStream_t s) {
    residual_norm_stats_kernel<T><<<row_blocks(p.R), 128, 0, s>>>(p);
    residual_norm_bwd_kernel<T><<<dim3(kRuns, (p.D + 255) / 256), 256, 0, s>>>(p);
    float *part = p.ws + 2ll * p.R;
    const unsigned blocks = (unsigned)((p.D + 127) / 128);
    if (p.dweight) sum_parts_kernel<<<blocks, 128, 0, s>>>(part, kRuns, p.D, p.dweight);
    if (p.dscale) sum_parts_kernel<<<blocks, 128, 0, s>>>(part + (long long)kRuns * p.D, kRuns, p.D, p.dscale);
    return 0;
}

#define INSTANTIATE(T)                                                                \
    template int launch_norm_gate<T>(const NormGateParams &, cudaStream_t);           \
    template int launch_norm_gate_bwd<T>(const NormGateParams &, cudaStream_t);       \
    template int launch_residual_norm<T>(const ResidualNormParams &, cudaStream_t);   \
    template int launch_residual_norm_bwd<T>(const ResidualNormParams &, cudaStream_t);
INSTANTIATE(float)
INSTANTIATE(__nv_bfloat16)
#undef INSTANTIATE

}  // namespace falcon
