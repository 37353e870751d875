// k_scan.cu -- the gated linear recurrence (falcon_scan), its backward pass
// and its single-token step:
//   a_t = 1/(1+exp(-f_t)),  h_t = (reset_t ? 0 : a_t h_{t-1}) + (1-a_t) x_t.
//
// One thread per (sequence, channel) walks the tokens.
#include "common.cuh"
#include "kernels.h"
#include "params_layer.h"

namespace falcon {

namespace {

// a = sigmoid(f) and c = 1 - a, each to full relative accuracy: with e =
// exp(-|f|) <= 1 the larger of the two is 1/(1+e), the smaller e/(1+e).
__device__ __forceinline__ void gates(float f, float &a, float &c) {
    const float e = expf(-fabsf(f));
    const float big = 1.f / (1.f + e), small = e * big;
    a = f < 0.f ? small : big;
    c = f < 0.f ? big : small;
}

template <typename T>
__global__ void __launch_bounds__(128) scan_kernel(ScanParams p) {
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    if (i >= (long long)p.N * p.D) return;
    const int n = (int)(i / p.D), ch = (int)(i % p.D);
    const int nblk = (p.L + kScanBlock - 1) / kScanBlock;
    float h = p.init_state ? p.init_state[i] : 0.f;
    for (int t = 0; t < p.L; ++t) {
        const long long row = (long long)n * p.L + t;
        if (p.marks && t % kScanBlock == 0) p.marks[((long long)n * nblk + t / kScanBlock) * p.D + ch] = h;
        const float x = to_f32(static_cast<const T *>(p.x)[row * p.ldx + ch]);
        float a, c;
        gates(to_f32(static_cast<const T *>(p.f)[row * p.ldf + ch]), a, c);
        h = p.reset && p.reset[row] ? c * x : fmaf(a, h, c * x);
        if (p.out) static_cast<T *>(p.out)[row * p.D + ch] = from_f32<T>(h);
    }
    if (p.final_state) p.final_state[i] = h;
}

template <typename T>
__global__ void __launch_bounds__(128) scan_bwd_kernel(ScanBwdParams p) {
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    if (i >= (long long)p.N * p.D) return;
    const int n = (int)(i / p.D), ch = (int)(i % p.D);
    const int nblk = (p.L + kScanBlock - 1) / kScanBlock;
    float g = p.dstate ? p.dstate[i] : 0.f;
    for (int b = nblk - 1; b >= 0; --b) {
        const int t0 = b * kScanBlock, len = min(kScanBlock, p.L - t0);
        float before[kScanBlock];  // the state before each of the block's tokens
        float h = p.marks[((long long)n * nblk + b) * p.D + ch];
        for (int t = 0; t < len; ++t) {
            const long long row = (long long)n * p.L + t0 + t;
            const float x = to_f32(static_cast<const T *>(p.x)[row * p.ldx + ch]);
            float a, c;
            gates(to_f32(static_cast<const T *>(p.f)[row * p.ldf + ch]), a, c);
            const bool r = p.reset && p.reset[row];
            before[t] = r ? 0.f : h;
            h = r ? c * x : fmaf(a, h, c * x);
        }
        for (int t = len - 1; t >= 0; --t) {
            const long long row = (long long)n * p.L + t0 + t;
            const float x = to_f32(static_cast<const T *>(p.x)[row * p.ldx + ch]);
            float a, c;
            gates(to_f32(static_cast<const T *>(p.f)[row * p.ldf + ch]), a, c);
            g += to_f32(static_cast<const T *>(p.dout)[row * p.D + ch]);
            static_cast<T *>(p.dx)[row * p.lddx + ch] = from_f32<T>(g * c);
            static_cast<T *>(p.df)[row * p.lddf + ch] = from_f32<T>(g * (before[t] - x) * (a * c));
            g = p.reset && p.reset[row] ? 0.f : a * g;
        }
    }
    if (p.dinitial) p.dinitial[i] = g;
}

template <typename T>
__global__ void __launch_bounds__(128) scan_step_kernel(ScanStepParams p) {
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    if (i >= (long long)p.N * p.D) return;
    const int n = (int)(i / p.D), ch = (int)(i % p.D);
    float a, c;
    gates(to_f32(static_cast<const T *>(p.f)[n * p.ldf + ch]), a, c);
    const float h = fmaf(a, p.state[i], c * to_f32(static_cast<const T *>(p.x)[n * p.ldx + ch]));
    p.state_out[i] = h;
    static_cast<T *>(p.out)[i] = from_f32<T>(h);
}

unsigned blocks(long long items) { return (unsigned)((items + 127) / 128); }

}  // namespace

template <typename T> int launch_scan(const ScanParams &p, cudaStream_t s) {
    scan_kernel<T><<<blocks((long long)p.N * p.D), 128, 0, s>>>(p);
    return 0;
}
template <typename T> int launch_scan_bwd(const ScanBwdParams &p, cudaStream_t s) {
    scan_bwd_kernel<T><<<blocks((long long)p.N * p.D), 128, 0, s>>>(p);
    return 0;
}
template <typename T> int launch_scan_step(const ScanStepParams &p, cudaStream_t s) {
    scan_step_kernel<T><<<blocks((long long)p.N * p.D), 128, 0, s>>>(p);
    return 0;
}

template int launch_scan<float>(const ScanParams &, cudaStream_t);
template int launch_scan<__nv_bfloat16>(const ScanParams &, cudaStream_t);
template int launch_scan_bwd<float>(const ScanBwdParams &, cudaStream_t);
template int launch_scan_bwd<__nv_bfloat16>(const ScanBwdParams &, cudaStream_t);
template int launch_scan_step<float>(const ScanStepParams &, cudaStream_t);
template int launch_scan_step<__nv_bfloat16>(const ScanStepParams &, cudaStream_t);

}  // namespace falcon
