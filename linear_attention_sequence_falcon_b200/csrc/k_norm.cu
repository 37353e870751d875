// k_norm.cu -- the norms around a block: falcon_norm_gate (behind it, with
// its gate) and falcon_residual_norm (in front of it, with the residual add),
// forward and backward.
//
//   n = o r,  r = 1/sqrt(mean(o^2) + eps);   e = gradient of n
//   do = r (e - n mean(e n)) = r e - o (r^3 mean(e o))
// so both passes need one set of sums per row (o^2; backward e o too), after
// which every output follows from what the threads hold: one pass over the
// data, each array moved once.
//
// A row is held by `tpr` threads, VEC neighbouring channels in NC places each
// (16-byte accesses where the arrays allow, single elements otherwise), so a
// thread keeps its channels from row to row: the weights stay in registers
// and their gradients are added up there, over the rows that the thread
// meets, then over the block's rows through shared memory, then over the
// blocks by sum_parts_kernel.  All orders are fixed by the sizes.  The next
// row's loads are issued before the present row's sums are joined.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "params_layer.h"

namespace falcon {

namespace {

constexpr int kSms = 148;
constexpr int kMinRows = 4;     // rows that a block walks at least, where weights' gradients are wanted
constexpr int kSegments = 8;    // partial sums joined side by side

// 1/sqrt(ms + eps); a row of zeros with eps = 0 is left as zeros
__device__ __forceinline__ float inv_rms(float ms, float eps) {
    const float v = ms + eps;
    return v == 0.f ? 0.f : rsqrtf(v);
}

// 1/(1+exp(-z)), to 0 for a far negative z
__device__ __forceinline__ float sigmoid(float z) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
    return s;
}

// ---- a thread's share of a row: NC places of VEC channels, as stored
template <typename T, int VEC> struct Piece;
template <> struct Piece<__nv_bfloat16, 8> { uint4 v; };
template <> struct Piece<float, 4> { uint4 v; };
template <> struct Piece<__nv_bfloat16, 1> { unsigned short v; };
template <> struct Piece<float, 1> { float v; };

__device__ __forceinline__ void widen(const Piece<__nv_bfloat16, 8> &p, float *f) {
    const uint32_t w[4] = {p.v.x, p.v.y, p.v.z, p.v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void widen(const Piece<float, 4> &p, float *f) {
    f[0] = __uint_as_float(p.v.x);
    f[1] = __uint_as_float(p.v.y);
    f[2] = __uint_as_float(p.v.z);
    f[3] = __uint_as_float(p.v.w);
}
__device__ __forceinline__ void widen(const Piece<__nv_bfloat16, 1> &p, float *f) {
    f[0] = __uint_as_float((uint32_t)p.v << 16);
}
__device__ __forceinline__ void widen(const Piece<float, 1> &p, float *f) { f[0] = p.v; }

__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ void narrow(Piece<__nv_bfloat16, 8> &p, const float *f) {
    p.v = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ void narrow(Piece<float, 4> &p, const float *f) {
    p.v = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ void narrow(Piece<__nv_bfloat16, 1> &p, const float *f) {
    p.v = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
}
__device__ __forceinline__ void narrow(Piece<float, 1> &p, const float *f) { p.v = f[0]; }

template <typename T, int VEC, int NC> struct Share {
    using P = Piece<T, VEC>;
    P p[NC];
    __device__ __forceinline__ void load(const T *row, int t, int tpr, int d, bool ok) {
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int c = (j * tpr + t) * VEC;
            p[j].v = {};
            if (ok && c < d) p[j] = *reinterpret_cast<const P *>(row + c);
        }
    }
    __device__ __forceinline__ void get(float *f) const {
#pragma unroll
        for (int j = 0; j < NC; ++j) widen(p[j], f + j * VEC);
    }
    static __device__ __forceinline__ void store(T *row, int t, int tpr, int d, const float *f) {
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int c = (j * tpr + t) * VEC;
            P q;
            narrow(q, f + j * VEC);
            if (c < d) *reinterpret_cast<P *>(row + c) = q;
        }
    }
};

// a thread's channels of an fp32 vector (NULL: ones); 0 behind the row's end
template <int VEC, int NC>
__device__ __forceinline__ void load_weights(float *w, const float *p, int t, int tpr, int d) {
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = (j * tpr + t) * VEC + i;
            w[j * VEC + i] = c < d ? (p ? p[c] : 1.f) : 0.f;
        }
}

// ---- sums over the threads of a row: shuffles inside a warp; more warps
// join through shared memory, one named barrier per row, the two halves of
// `red` in turn
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], int tpr, int slot, float (*red)[32][2], int parity) {
    for (int o = min(tpr, 32) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (tpr <= 32) return;
    const int warp = threadIdx.x >> 5, per = tpr >> 5, first = slot * per;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) red[parity][warp][k] = v[k];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + slot), "r"(tpr) : "memory");
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
    for (int i = 0; i < per; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += red[parity][first + i][k];
}

// ---- a thread's sums over its rows, joined over the block's slots and
// written as the block's partial sum part[0..d)
template <int VEC, int NC>
__device__ __forceinline__ void block_part(float *acc, int t, int tpr, int slot, int slots, int d, float *part,
                                           float *buf) {
    constexpr int E = VEC * NC;
    // the slots of one warp first
    for (int o = tpr; o < 32; o <<= 1)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
    const int lines = tpr < 32 ? blockDim.x >> 5 : slots;    // sums left per channel
    const int line = tpr < 32 ? threadIdx.x >> 5 : slot;
    const bool holds = tpr >= 32 || (threadIdx.x & 31) < tpr;
    if (lines > 1) {
        __syncthreads();
        if (holds && line > 0)
#pragma unroll
            for (int e = 0; e < E; ++e) buf[((line - 1) * E + e) * tpr + t] = acc[e];
        __syncthreads();
        if (line > 0) return;
        for (int i = 0; i < lines - 1; ++i)
            if (holds)
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += buf[(i * E + e) * tpr + t];
    }
    if (!holds) return;
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = (j * tpr + t) * VEC + i;
            if (c < d) part[c] = acc[j * VEC + i];
        }
}

// ---- the rows of the gated norm: (b, l, h) with h innermost, or, where a
// block stays with one head, (b, l)
struct GateRows {
    long long o, g, out, d_o, dg;  // offsets of the row's first channel
    int b, l, h;                   // h counts inside `heads`
};

__device__ __forceinline__ void gate_offsets(const NormGateParams &p, GateRows &r, int h) {
    const long long token = (long long)r.b * p.L + r.l;
    r.o = r.b * p.o_sb + h * p.o_sh + r.l * p.o_sl;
    r.d_o = r.b * p.do_sb + h * p.do_sh + r.l * p.do_sl;
    r.out = (token * p.H + h) * p.d;
    r.g = token * p.ldg + (long long)h * p.d;
    r.dg = token * p.lddg + (long long)h * p.d;
}

struct GateWalk {
    int heads, h0;                 // heads that the rows run over, from h0
    long long rows, row, step;
    int db, dl, dh;                // the step in rows, taken apart
    __device__ __forceinline__ void begin(const NormGateParams &p, int parts, int slots, int slot, GateRows &r) {
        heads = p.per_head ? 1 : p.H;
        h0 = p.per_head ? blockIdx.x / parts : 0;
        rows = (long long)p.B * p.L * heads;
        row = (long long)(blockIdx.x % parts) * slots + slot;
        step = (long long)parts * slots;
        dh = (int)(step % heads);
        const long long dt = step / heads;
        dl = (int)(dt % p.L);
        db = (int)(dt / p.L);
        r.h = (int)(row % heads);
        const long long token = row / heads;
        r.l = (int)(token % p.L);
        r.b = (int)(token / p.L);
    }
    __device__ __forceinline__ void next(const NormGateParams &p, GateRows &r) {
        row += step;
        r.h += dh;
        r.l += dl;
        r.b += db;
        if (r.h >= heads) { r.h -= heads; ++r.l; }
        if (r.l >= p.L) { r.l -= p.L; ++r.b; }
    }
};

template <typename T, int VEC, int NC, int MT, bool GATE>
__global__ void __launch_bounds__(MT, MT == 256 ? 4 : 1) norm_gate_kernel(NormGateParams p, int tpr, int parts) {
    constexpr int E = VEC * NC;
    using S = Share<T, VEC, NC>;
    __shared__ float red[2][32][2];
    const int t = threadIdx.x % tpr, slot = threadIdx.x / tpr, slots = blockDim.x / tpr, d = p.d;
    GateRows r;
    GateWalk w;
    w.begin(p, parts, slots, slot, r);
    float wt[E];
    load_weights<VEC, NC>(wt, p.weight ? p.weight + (long long)w.h0 * d : nullptr, t, tpr, d);
    S o, z;
    auto fetch = [&]() {
        const bool ok = w.row < w.rows;
        if (ok) gate_offsets(p, r, w.h0 + r.h);
        o.load(static_cast<const T *>(p.o) + r.o, t, tpr, d, ok);
        if constexpr (GATE) z.load(static_cast<const T *>(p.gate) + r.g, t, tpr, d, ok);
    };
    r.o = r.g = r.out = 0;
    fetch();
    const long long first = (long long)(blockIdx.x % parts) * slots;
    int parity = 0;
    for (long long base = first; base < w.rows; base += w.step, parity ^= 1) {
        float ov[E], zv[E], sum[1] = {0.f};
        o.get(ov);
        if constexpr (GATE) z.get(zv);
        const bool ok = w.row < w.rows;
        T *out = static_cast<T *>(p.out) + r.out;
#pragma unroll
        for (int e = 0; e < E; ++e) sum[0] = fmaf(ov[e], ov[e], sum[0]);
        w.next(p, r);
        fetch();
        row_sum<1>(sum, tpr, slot, red, parity);
        const float rstd = inv_rms(sum[0] / d, p.eps);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            ov[e] *= rstd * wt[e];
            if constexpr (GATE) ov[e] *= zv[e] * sigmoid(zv[e]);
        }
        if (ok) S::store(out, t, tpr, d, ov);
    }
}

template <typename T, int VEC, int NC, int MT, bool GATE>
__global__ void __launch_bounds__(MT, MT == 256 ? 2 : 1) norm_gate_bwd_kernel(NormGateParams p, int tpr, int parts) {
    constexpr int E = VEC * NC;
    using S = Share<T, VEC, NC>;
    __shared__ float red[2][32][2];
    __shared__ float buf[MT == 256 ? 256 * E : 1];
    const int t = threadIdx.x % tpr, slot = threadIdx.x / tpr, slots = blockDim.x / tpr, d = p.d;
    GateRows r;
    GateWalk w;
    w.begin(p, parts, slots, slot, r);
    float wt[E], dw[E];
    load_weights<VEC, NC>(wt, p.weight ? p.weight + (long long)w.h0 * d : nullptr, t, tpr, d);
#pragma unroll
    for (int e = 0; e < E; ++e) dw[e] = 0.f;
    S o, z, g;
    auto fetch = [&]() {
        const bool ok = w.row < w.rows;
        if (ok) gate_offsets(p, r, w.h0 + r.h);
        o.load(static_cast<const T *>(p.o) + r.o, t, tpr, d, ok);
        g.load(static_cast<const T *>(p.dout) + r.out, t, tpr, d, ok);
        if constexpr (GATE) z.load(static_cast<const T *>(p.gate) + r.g, t, tpr, d, ok);
    };
    r.o = r.g = r.out = r.d_o = r.dg = 0;
    fetch();
    const long long first = (long long)(blockIdx.x % parts) * slots;
    const float inv_d = 1.f / d;
    int parity = 0;
    for (long long base = first; base < w.rows; base += w.step, parity ^= 1) {
        float ov[E], zv[E], gv[E], sum[2] = {0.f, 0.f};
        o.get(ov);
        g.get(gv);
        if constexpr (GATE) z.get(zv);
        const bool ok = w.row < w.rows;
        T *d_o = static_cast<T *>(p.d_o) + r.d_o, *dgate = static_cast<T *>(p.dgate) + r.dg;
        // gv: dout -> e = dout s(z); zv: z -> dout w s'(z) o, still without r
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if constexpr (GATE) {
                const float s = sigmoid(zv[e]), act = zv[e] * s, dy = gv[e];
                gv[e] = dy * act;
                zv[e] = dy * wt[e] * ov[e] * (s + act * (1.f - s));
            }
            sum[0] = fmaf(ov[e], ov[e], sum[0]);
            sum[1] = fmaf(gv[e] * wt[e], ov[e], sum[1]);
        }
        w.next(p, r);
        fetch();
        row_sum<2>(sum, tpr, slot, red, parity);
        const float rstd = inv_rms(sum[0] * inv_d, p.eps);
        const float m = sum[1] * inv_d * rstd * rstd;  // mean(e w n) r
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float n = ov[e] * rstd;
            dw[e] = fmaf(gv[e], n, dw[e]);
            ov[e] = fmaf(-ov[e], m, gv[e] * wt[e]) * rstd;
            if constexpr (GATE) zv[e] *= rstd;
        }
        if (ok) {
            S::store(d_o, t, tpr, d, ov);
            if constexpr (GATE) S::store(dgate, t, tpr, d, zv);
        }
    }
    if (p.dweight)
        block_part<VEC, NC>(dw, t, tpr, slot, slots, d,
                            p.ws + ((long long)(blockIdx.x % parts) * (p.per_head ? p.H : 1) + w.h0) * d, buf);
}

template <typename T, int VEC, int NC, int MT, bool ADD>
__global__ void __launch_bounds__(MT, MT == 256 ? 4 : 1) residual_norm_kernel(ResidualNormParams p, int tpr) {
    constexpr int E = VEC * NC;
    using S = Share<T, VEC, NC>;
    __shared__ float red[2][32][2];
    const int t = threadIdx.x % tpr, slot = threadIdx.x / tpr, slots = blockDim.x / tpr, d = p.D;
    float wt[E], sc[E];
    load_weights<VEC, NC>(wt, p.weight, t, tpr, d);
    if constexpr (ADD) load_weights<VEC, NC>(sc, p.scale, t, tpr, d);
    const int step = gridDim.x * slots;
    long long row = (long long)blockIdx.x * slots + slot;
    S a, b;
    auto fetch = [&]() {
        const long long at = row < p.R ? row * d : 0;
        a.load(static_cast<const T *>(p.r) + at, t, tpr, d, row < p.R);
        if constexpr (ADD) b.load(static_cast<const T *>(p.y) + at, t, tpr, d, row < p.R);
    };
    fetch();
    int parity = 0;
    for (long long base = (long long)blockIdx.x * slots; base < p.R; base += step, parity ^= 1) {
        float v[E], y[E], sum[1] = {0.f};
        a.get(v);
        if constexpr (ADD) b.get(y);
        const bool ok = row < p.R;
        const long long at = row * d;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if constexpr (ADD) v[e] = fmaf(sc[e], y[e], v[e]);
            sum[0] = fmaf(v[e], v[e], sum[0]);
        }
        row += step;
        fetch();
        row_sum<1>(sum, tpr, slot, red, parity);
        const float rstd = inv_rms(sum[0] / d, p.eps);
        if (ok && p.r_out) S::store(static_cast<T *>(p.r_out) + at, t, tpr, d, v);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= rstd * wt[e];
        if (ok) S::store(static_cast<T *>(p.h) + at, t, tpr, d, v);
    }
}

template <typename T, int VEC, int NC, int MT, bool ADD>
__global__ void __launch_bounds__(MT, MT == 256 ? 2 : 1) residual_norm_bwd_kernel(ResidualNormParams p, int tpr) {
    constexpr int E = VEC * NC;
    using S = Share<T, VEC, NC>;
    __shared__ float red[2][32][2];
    __shared__ float buf[MT == 256 ? 256 * E : 1];
    const int t = threadIdx.x % tpr, slot = threadIdx.x / tpr, slots = blockDim.x / tpr, d = p.D;
    float wt[E], sc[E], dw[E], ds[E];
    load_weights<VEC, NC>(wt, p.weight, t, tpr, d);
    load_weights<VEC, NC>(sc, p.scale, t, tpr, d);
#pragma unroll
    for (int e = 0; e < E; ++e) dw[e] = ds[e] = 0.f;
    const int step = gridDim.x * slots;
    long long row = (long long)blockIdx.x * slots + slot;
    S a, b, g, s;  // r_out, y, dh, dr_out
    const bool stream = p.dr_out != nullptr;
    auto fetch = [&]() {
        const bool ok = row < p.R;
        const long long at = ok ? row * d : 0;
        a.load(static_cast<const T *>(p.r) + at, t, tpr, d, ok);
        g.load(static_cast<const T *>(p.dh) + at, t, tpr, d, ok);
        s.load(static_cast<const T *>(p.dr_out) + at, t, tpr, d, ok && stream);
        if constexpr (ADD) b.load(static_cast<const T *>(p.y) + at, t, tpr, d, ok);
    };
    fetch();
    const float inv_d = 1.f / d;
    int parity = 0;
    for (long long base = (long long)blockIdx.x * slots; base < p.R; base += step, parity ^= 1) {
        const S ca = a, cg = g, cs = s, cb = b;  // as stored: widened again behind the sums
        float sum[2] = {0.f, 0.f};
        {
            float v[E], e_[E];
            ca.get(v);
            cg.get(e_);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                sum[0] = fmaf(v[e], v[e], sum[0]);
                sum[1] = fmaf(e_[e] * wt[e], v[e], sum[1]);
            }
        }
        const bool ok = row < p.R;
        const long long at = row * d;
        row += step;
        fetch();
        row_sum<2>(sum, tpr, slot, red, parity);
        const float rstd = inv_rms(sum[0] * inv_d, p.eps);
        const float m = sum[1] * inv_d * rstd * rstd;  // mean(e n) r
        float v[E], x[E];
        ca.get(v);
        cg.get(x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            dw[e] = fmaf(x[e], v[e] * rstd, dw[e]);
            x[e] = fmaf(-v[e], m, x[e] * wt[e]) * rstd;
        }
        cs.get(v);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] += v[e];
        if constexpr (ADD) {
            cb.get(v);
#pragma unroll
            for (int e = 0; e < E; ++e) ds[e] = fmaf(x[e], v[e], ds[e]);
        }
        if (ok) {
            S::store(static_cast<T *>(p.dr) + at, t, tpr, d, x);
            if (p.dy) {
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] *= sc[e];
                S::store(static_cast<T *>(p.dy) + at, t, tpr, d, x);
            }
        }
    }
    if (p.dweight) block_part<VEC, NC>(dw, t, tpr, slot, slots, d, p.ws + (long long)blockIdx.x * d, buf);
    if constexpr (ADD)
        if (p.dscale)
            block_part<VEC, NC>(ds, t, tpr, slot, slots, d, p.ws + ((long long)gridDim.x + blockIdx.x) * d, buf);
}

// out[c] = sum over i of part[i*n + c]: 32 channels per block, kSegments runs
// of partial sums side by side, joined in order; blockIdx.y takes the second
// set of partial sums (behind the first) and its output
__global__ void __launch_bounds__(32 * kSegments) sum_parts_kernel(const float *part, int parts, long long n,
                                                                   float *out0, float *out1) {
    __shared__ float seg[kSegments][32];
    float *out = blockIdx.y ? out1 : out0;
    const long long c = (long long)blockIdx.x * 32 + threadIdx.x % 32;
    const int s = threadIdx.x / 32;
    const float *at = part + (long long)blockIdx.y * parts * n;
    float acc = 0.f;
    if (out && c < n)
#pragma unroll 8
        for (int i = s; i < parts; i += kSegments) acc += at[i * n + c];
    seg[s][threadIdx.x % 32] = acc;
    __syncthreads();
    if (s != 0 || !out || c >= n) return;
#pragma unroll
    for (int i = 1; i < kSegments; ++i) acc += seg[i][threadIdx.x];
    out[c] = acc;
}

// ---- launches

// How a row of d channels is laid on threads: 8 channels a thread (16 beyond
// 8192), so that the accumulators of the weights' gradients stay in registers.
struct Layout {
    int tpr, threads, slots, per_sm;
    bool wide;  // 16 channels a thread
    explicit Layout(int d) {
        wide = d > 8192;
        const int need = (d + (wide ? 15 : 7)) / (wide ? 16 : 8);
        if (need > 32) {
            tpr = (need + 31) / 32 * 32;
        } else {
            tpr = 1;
            while (tpr < need) tpr *= 2;
        }
        slots = tpr >= 256 ? 1 : 256 / tpr;
        threads = tpr * slots;
        per_sm = threads > 1024 ? 1 : 1024 / threads;
    }
    // blocks for `rows` rows, at least `least` rows each where there are as many
    int blocks(long long rows, int least) const {
        const long long want = (rows + (long long)slots * least - 1) / ((long long)slots * least);
        return (int)(want < (long long)kSms * per_sm ? want : (long long)kSms * per_sm);
    }
};

bool vec_ok(const void *p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// go(VEC, NC, threads' limit): 16-byte pieces where `vec`, else single elements
template <typename T, typename F> int with_layout(const Layout &lay, bool vec, F go) {
    constexpr int V = 16 / sizeof(T), N = 8 / V;
    using std::integral_constant;
    if (lay.wide)
        return vec ? go(integral_constant<int, V>(), integral_constant<int, 2 * N>(), integral_constant<int, 1024>())
                   : go(integral_constant<int, 1>(), integral_constant<int, 16>(), integral_constant<int, 1024>());
    if (lay.threads > 256)
        return vec ? go(integral_constant<int, V>(), integral_constant<int, N>(), integral_constant<int, 1024>())
                   : go(integral_constant<int, 1>(), integral_constant<int, 8>(), integral_constant<int, 1024>());
    return vec ? go(integral_constant<int, V>(), integral_constant<int, N>(), integral_constant<int, 256>())
               : go(integral_constant<int, 1>(), integral_constant<int, 8>(), integral_constant<int, 256>());
}

template <typename T> bool gate_vec(const NormGateParams &p) {
    const int v = 16 / sizeof(T);
    return p.d % v == 0 && p.o_sb % v == 0 && p.o_sh % v == 0 && p.o_sl % v == 0 && vec_ok(p.o) &&
           vec_ok(p.gate) && (!p.gate || p.ldg % v == 0);
}

int gate_parts(const Layout &lay, const NormGateParams &p, int least) {
    const long long rows = (long long)p.B * p.L * (p.per_head ? 1 : p.H);
    if (!p.per_head) return lay.blocks(rows, least);
    // every head has blocks of its own: share the device's between them
    const int all = lay.blocks(rows, least), share = (kSms * lay.per_sm + p.H - 1) / p.H;
    return all < share ? all : share;
}

}  // namespace

size_t norm_gate_bwd_ws_bytes(int, int B, int H, int L, int d) {
    const Layout lay(d);
    NormGateParams p{};
    p.B = B; p.H = H; p.L = L;
    size_t most = 0;
    for (p.per_head = 0; p.per_head < 2; ++p.per_head) {
        const size_t n = (size_t)gate_parts(lay, p, kMinRows) * (p.per_head ? H : 1) * d;
        most = n > most ? n : most;
    }
    return sizeof(float) * most;
}
size_t residual_norm_bwd_ws_bytes(int, int R, int D) {
    return sizeof(float) * 2 * (size_t)Layout(D).blocks(R, kMinRows) * D;
}

template <typename T> int launch_norm_gate(const NormGateParams &p, cudaStream_t s) {
    const Layout lay(p.d);
    const bool vec = gate_vec<T>(p) && vec_ok(p.out);
    const int parts = gate_parts(lay, p, 1);
    const unsigned grid = (unsigned)parts * (p.per_head ? p.H : 1);
    return with_layout<T>(lay, vec, [&](auto v, auto nc, auto mt) {
        if (p.gate)
            norm_gate_kernel<T, v(), nc(), mt(), true><<<grid, lay.threads, 0, s>>>(p, lay.tpr, parts);
        else
            norm_gate_kernel<T, v(), nc(), mt(), false><<<grid, lay.threads, 0, s>>>(p, lay.tpr, parts);
        return 0;
    });
}

template <typename T> int launch_norm_gate_bwd(const NormGateParams &p, cudaStream_t s) {
    const Layout lay(p.d);
    const int v16 = 16 / sizeof(T);
    const bool vec = gate_vec<T>(p) && vec_ok(p.dout) && vec_ok(p.d_o) &&
                     vec_ok(p.dgate) && p.do_sb % v16 == 0 && p.do_sh % v16 == 0 && p.do_sl % v16 == 0 &&
                     (!p.dgate || p.lddg % v16 == 0);
    const int parts = gate_parts(lay, p, kMinRows);
    const unsigned grid = (unsigned)parts * (p.per_head ? p.H : 1);
    with_layout<T>(lay, vec, [&](auto v, auto nc, auto mt) {
        if (p.gate)
            norm_gate_bwd_kernel<T, v(), nc(), mt(), true><<<grid, lay.threads, 0, s>>>(p, lay.tpr, parts);
        else
            norm_gate_bwd_kernel<T, v(), nc(), mt(), false><<<grid, lay.threads, 0, s>>>(p, lay.tpr, parts);
        return 0;
    });
    if (!p.dweight) return 0;
    const long long n = (long long)p.d * (p.per_head ? p.H : 1);
    sum_parts_kernel<<<(unsigned)((n + 31) / 32), 32 * kSegments, 0, s>>>(p.ws, parts, n, p.dweight, nullptr);
    return 0;
}

template <typename T> int launch_residual_norm(const ResidualNormParams &p, cudaStream_t s) {
    const Layout lay(p.D);
    const bool vec = p.D % (16 / (int)sizeof(T)) == 0 && vec_ok(p.r) && vec_ok(p.y) &&
                     vec_ok(p.r_out) && vec_ok(p.h);
    const unsigned grid = (unsigned)lay.blocks(p.R, 1);
    return with_layout<T>(lay, vec, [&](auto v, auto nc, auto mt) {
        if (p.y)
            residual_norm_kernel<T, v(), nc(), mt(), true><<<grid, lay.threads, 0, s>>>(p, lay.tpr);
        else
            residual_norm_kernel<T, v(), nc(), mt(), false><<<grid, lay.threads, 0, s>>>(p, lay.tpr);
        return 0;
    });
}

template <typename T> int launch_residual_norm_bwd(const ResidualNormParams &p, cudaStream_t s) {
    const Layout lay(p.D);
    const bool vec = p.D % (16 / (int)sizeof(T)) == 0 && vec_ok(p.r) && vec_ok(p.y) &&
                     vec_ok(p.dh) && vec_ok(p.dr_out) && vec_ok(p.dr) &&
                     vec_ok(p.dy);
    const unsigned grid = (unsigned)lay.blocks(p.R, kMinRows);
    with_layout<T>(lay, vec, [&](auto v, auto nc, auto mt) {
        if (p.y)
            residual_norm_bwd_kernel<T, v(), nc(), mt(), true><<<grid, lay.threads, 0, s>>>(p, lay.tpr);
        else
            residual_norm_bwd_kernel<T, v(), nc(), mt(), false><<<grid, lay.threads, 0, s>>>(p, lay.tpr);
        return 0;
    });
    if (p.dweight || p.dscale)
        sum_parts_kernel<<<dim3((unsigned)((p.D + 31) / 32), p.dscale ? 2 : 1), 32 * kSegments, 0, s>>>(
            p.ws, (int)grid, p.D, p.dweight, p.dscale);
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
