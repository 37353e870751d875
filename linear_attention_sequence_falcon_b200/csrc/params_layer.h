// params_layer.h -- the parameter blocks the C ABI (api_layer.cu) hands to
// the layer operators' kernels (k_scan.cu, k_norm.cu).  Not installed; the
// public boundary is include/falcon.h.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace falcon {

constexpr int kScanBlock = 64;     // tokens between two marks (FALCON_SCAN_BLOCK)
constexpr int kNormMaxD = 16384;   // the longest row of the norms (FALCON_NORM_MAX_D)

struct ScanParams {
    int N, L, D;
    long long ldx, ldf;            // elements from one token to the next
    const void *x, *f;
    const unsigned char *reset;    // [N,L] or NULL
    const float *init_state;       // [N,D] or NULL
    void *out;                     // [N,L,D], or NULL (marks only)
    float *final_state, *marks;    // each may be NULL
};

struct ScanBwdParams {
    int N, L, D;
    long long ldx, ldf, lddx, lddf;
    const void *x, *f;
    const unsigned char *reset;
    const float *marks;            // [N,ceil(L/kScanBlock),D]
    const void *dout;
    const float *dstate;           // may be NULL
    void *dx, *df;
    float *dinitial;               // may be NULL
};

struct ScanStepParams {
    int N, D;
    long long ldx, ldf;
    const void *x, *f;
    const float *state;
    float *state_out;
    void *out;
};

// Division by a fixed number below 2^31 of numbers below 2^31: one product.
struct FastDiv {
    unsigned by, factor, shift;
};

struct NormGateParams {
    int B, H, L, d, per_head;
    int small;                     // fewer than 2^31 rows, every offset below 2^31: the divisions below hold
    FastDiv heads, tokens;         // rows into (token, head), tokens into (b, l); set by the launcher
    long long o_sb, o_sh, o_sl, ldg;
    float eps;
    const void *o, *gate;          // gate may be NULL
    const float *weight;           // may be NULL
    void *out;
    // backward
    const void *dout;
    void *d_o, *dgate;
    long long do_sb, do_sh, do_sl, lddg;
    float *dweight;                // may be NULL
    float *ws;
};

struct ResidualNormParams {
    int R, D;
    float eps;
    const void *r, *y;             // forward: the stream and what is added (may be NULL); backward: r_out and y
    const float *scale, *weight;   // each may be NULL
    void *r_out, *h;
    // backward
    const void *dh, *dr_out;       // dr_out may be NULL
    void *dr, *dy;                 // dy may be NULL
    float *dscale, *dweight;       // each may be NULL
    float *ws;
};

template <typename T> int launch_scan(const ScanParams &p, cudaStream_t s);
template <typename T> int launch_scan_bwd(const ScanBwdParams &p, cudaStream_t s);
// the same for more than 32 channels (k_scan_tile.cu): fp32 rows on 16-byte
// boundaries, bf16 rows on any; 1 (nothing launched) for what they do not cover
template <typename T> int launch_scan_tile(const ScanParams &p, cudaStream_t s);
template <typename T> int launch_scan_bwd_tile(const ScanBwdParams &p, cudaStream_t s);
unsigned int scan_tile_wait_timeouts();
template <typename T> int launch_scan_step(const ScanStepParams &p, cudaStream_t s);
template <typename T> int launch_norm_gate(const NormGateParams &p, cudaStream_t s);
template <typename T> int launch_norm_gate_bwd(const NormGateParams &p, cudaStream_t s);
template <typename T> int launch_residual_norm(const ResidualNormParams &p, cudaStream_t s);
template <typename T> int launch_residual_norm_bwd(const ResidualNormParams &p, cudaStream_t s);
// bytes of the backward passes' workspaces (p.ws)
size_t norm_gate_bwd_ws_bytes(int bf16, int B, int H, int L, int d);
size_t residual_norm_bwd_ws_bytes(int bf16, int R, int D);

}  // namespace falcon
