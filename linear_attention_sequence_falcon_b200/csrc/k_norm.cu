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
// (16-byte accesses where the arrays allow, two bf16 or single elements
// otherwise), so a thread keeps its channels from row to row: the weights stay
// in registers and their gradients are added up there, over the rows that the
// thread meets, then over the block's rows through shared memory, then over
// the blocks by sum_parts_kernel.  All orders are fixed by the sizes.
//
// The bound is HBM: what it takes is bytes in flight.  A thread keeps the next
// two rows' pieces on their way as asynchronous copies into its own places
// of shared memory (no other thread reads them, so no barrier is needed, and
// no registers are held).
#include <algorithm>
#include <atomic>
#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "params_layer.h"

namespace falcon {

namespace {

constexpr int kSms = 148;
constexpr int kMinRows = 4;     // rows that a thread walks at least, where weights' gradients are wanted
                                // and the device is full
constexpr int kSegments = 32;   // partial sums joined side by side
constexpr int kMaxRows = 3;     // rows of a thread in shared memory: the present one and two on their way

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

// ---- VEC neighbouring channels, as stored
template <typename T, int VEC> struct Piece;
template <> struct Piece<__nv_bfloat16, 8> { uint4 v; };
template <> struct Piece<__nv_bfloat16, 2> { uint32_t v; };
template <> struct Piece<__nv_bfloat16, 1> { unsigned short v; };
template <> struct Piece<float, 4> { uint4 v; };
template <> struct Piece<float, 1> { uint32_t v; };

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ void widen(const Piece<__nv_bfloat16, 8> &p, float *f) {
    f[0] = low(p.v.x), f[1] = high(p.v.x), f[2] = low(p.v.y), f[3] = high(p.v.y);
    f[4] = low(p.v.z), f[5] = high(p.v.z), f[6] = low(p.v.w), f[7] = high(p.v.w);
}
__device__ __forceinline__ void widen(const Piece<__nv_bfloat16, 2> &p, float *f) { f[0] = low(p.v), f[1] = high(p.v); }
__device__ __forceinline__ void widen(const Piece<__nv_bfloat16, 1> &p, float *f) { f[0] = low(p.v); }
__device__ __forceinline__ void widen(const Piece<float, 4> &p, float *f) {
    f[0] = __uint_as_float(p.v.x), f[1] = __uint_as_float(p.v.y);
    f[2] = __uint_as_float(p.v.z), f[3] = __uint_as_float(p.v.w);
}
__device__ __forceinline__ void widen(const Piece<float, 1> &p, float *f) { f[0] = __uint_as_float(p.v); }

__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ void narrow(Piece<__nv_bfloat16, 8> &p, const float *f) {
    p.v = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ void narrow(Piece<__nv_bfloat16, 2> &p, const float *f) { p.v = pack2(f[0], f[1]); }
__device__ __forceinline__ void narrow(Piece<__nv_bfloat16, 1> &p, const float *f) {
    p.v = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
}
__device__ __forceinline__ void narrow(Piece<float, 4> &p, const float *f) {
    p.v = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ void narrow(Piece<float, 1> &p, const float *f) { p.v = __float_as_uint(f[0]); }

// ---- a thread's pieces of the present row and of those to come, A arrays each:
// S rows in shared memory (three where they fit the block's, whatever fits
// otherwise), S - 1 of them on their way.  Of single elements the next row's are
// loaded into registers: bf16 has no asynchronous copy of two bytes, and in fp32
// copies of four took longer (backward at 1003x1111 off 16 bytes, 16 against
// 14 us).  The widest fp32 rows have no room at all (S = 0) and are read when used.
//
// SHIFT: pieces of 16 bytes although rows do not start on them.  Where a row
// starts within its first piece repeats after VEC rows at most, so a thread that
// walks rows in steps of such a number finds it the same in each: `lead`
// elements of the row before, which are read and put to 0, and its channels stay
// its own.  (All arrays have the same rows here, and start on 16 bytes.)  The
// residual norm's backward pass of 16384 rows in bf16, against pieces of one
// element: 62 against 129 us of 1111 channels, 223 against 2303 us of 5001.
template <typename T, int VEC, int NC, int A, int MT, int BLOCKS, bool SHIFT = false> struct Ahead {
    using P = Piece<T, VEC>;
    static constexpr int kRow = A * NC * (int)sizeof(P);  // bytes per thread
    // rows that fit BLOCKS blocks of an SM; two if one block can have them
    static constexpr int kFit = 216 * 1024 / BLOCKS / (MT * kRow), kAlone = 200 * 1024 / (MT * kRow);
    static constexpr int kRows = kFit >= 2 ? kFit : kAlone < 2 ? kAlone : 2;
    static constexpr bool kHeld = VEC == 1;
    static constexpr int S = kHeld ? 0 : kRows < kMaxRows ? kRows : kMaxRows;
    static constexpr int kAhead = S > 0 ? S - 1 : kHeld ? 1 : 0;
    static constexpr int kBytes = S * kRow;
    P *mine;
    int t, tpr, d, threads, lead;
    const T *at[S == 0 && !kHeld ? A : 1];    // S = 0: the present row
    P held[kHeld ? A : 1][NC], next_[kHeld ? A : 1][NC];

    __device__ __forceinline__ Ahead(uint8_t *smem, int t_, int tpr_, int d_, int lead_ = 0)
        : mine(reinterpret_cast<P *>(smem) + threadIdx.x), t(t_), tpr(tpr_), d(d_), threads(blockDim.x),
          lead(SHIFT ? lead_ : 0) {
        static_assert(!SHIFT || (S > 0 && sizeof(P) == 16), "shifted rows pass through shared memory");
    }
    // the first channel of place j (before the row, where a shifted one begins)
    __device__ __forceinline__ int channel(int j) const { return (j * tpr + t) * VEC - (SHIFT ? lead : 0); }
    __device__ __forceinline__ P *place(int stage, int a, int j) const {
        return mine + ((stage * A + a) * NC + j) * threads;
    }
    // array a of a row (zeros where not ok, and behind the row's end)
    __device__ __forceinline__ void fetch(int stage, int a, const T *row, bool ok) {
        if constexpr (kHeld) {
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const int c = (j * tpr + t) * VEC;
                held[a][j] = next_[a][j];
                next_[a][j].v = 0;
                if (ok && c < d) next_[a][j] = *reinterpret_cast<const P *>(row + c);
            }
        } else if constexpr (S == 0) {
            at[a] = ok ? row : nullptr;
        } else {
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const int c = channel(j);
                const bool in = ok && c < d;
                const uint32_t dst = (uint32_t)__cvta_generic_to_shared(place(stage, a, j));
                const T *src = in ? row + c : SHIFT && ok ? row - lead : row;
                // (a piece that ends behind its row is read up to there, and filled with zeros)
                const int bytes = !in ? 0 : SHIFT ? min(VEC, d - c) * (int)sizeof(T) : (int)sizeof(P);
                if constexpr (sizeof(P) == 16)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
                else
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
            }
        }
    }
    static __device__ __forceinline__ void close() {
        if constexpr (S > 0) asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // all but the last kAhead rows' copies have come
    static __device__ __forceinline__ void wait() {
        if constexpr (S > 0) asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
    }
    static __device__ __forceinline__ void wait_all() {
        if constexpr (S > 0) asm volatile("cp.async.wait_all;" ::: "memory");
    }
    __device__ __forceinline__ void get(int stage, int a, float *f) const {
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            if constexpr (kHeld) {
                widen(held[a][j], f + j * VEC);
            } else if constexpr (S == 0) {
                const int c = (j * tpr + t) * VEC;
                P v{};
                if (at[a] && c < d) v = *reinterpret_cast<const P *>(at[a] + c);
                widen(v, f + j * VEC);
            } else {
                widen(*place(stage, a, j), f + j * VEC);
                if constexpr (SHIFT)
                    if (j == 0)
#pragma unroll
                        for (int i = 0; i < VEC; ++i) f[i] = channel(0) + i < 0 ? 0.f : f[i];
            }
        }
    }
    __device__ __forceinline__ void store(T *row, const float *f) const {
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int c = channel(j);
            P q;
            narrow(q, f + j * VEC);
            if (SHIFT && (c < 0 || c + VEC > d)) {  // the row's ends: element by element
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    Piece<T, 1> one;
                    narrow(one, f + j * VEC + i);
                    if (c + i >= 0 && c + i < d) *reinterpret_cast<Piece<T, 1> *>(row + c + i) = one;
                }
            } else if (c < d) {
                *reinterpret_cast<P *>(row + c) = q;
            }
        }
    }
    // the stage behind the present one's last copy, and the next present one
    static __device__ __forceinline__ int last(int stage) { return S <= 1 ? 0 : stage == 0 ? S - 1 : stage - 1; }
    static __device__ __forceinline__ int next(int stage) { return S <= 1 || stage == S - 1 ? 0 : stage + 1; }
};

// VEC channels c.. of an fp32 vector may be moved in 16-byte accesses.  One by
// one, a warp's access touches a sector for each lane, VEC times: of few rows
// that was half of the time (residual norm backward in bf16, 9x8192: 17.0
// against 9.7 us; 1003x4096: 25 against 18).
template <int VEC> __device__ __forceinline__ bool fours(const float *p, int c, int d) {
    return VEC % 4 == 0 && c >= 0 && c + VEC <= d && (reinterpret_cast<uintptr_t>(p + c) & 15u) == 0;
}

// a thread's channels of an fp32 vector (NULL: ones); 0 outside of the row
template <int VEC, int NC, bool FOURS = true>
__device__ __forceinline__ void load_weights(float *w, const float *p, int t, int tpr, int d, int lead = 0) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int c = (j * tpr + t) * VEC - lead;
        if (FOURS && p && fours<VEC>(p, c, d)) {
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i) {
                const float4 four = reinterpret_cast<const float4 *>(p + c)[i];
                w[j * VEC + 4 * i] = four.x, w[j * VEC + 4 * i + 1] = four.y;
                w[j * VEC + 4 * i + 2] = four.z, w[j * VEC + 4 * i + 3] = four.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                w[j * VEC + i] = c + i >= 0 && c + i < d ? (p ? p[c + i] : 1.f) : 0.f;
        }
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
    for (int j = 0; j < NC; ++j) {
        const int c = (j * tpr + t) * VEC;
        if (fours<VEC>(part, c, d)) {
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i) {
                const float *a = acc + j * VEC + 4 * i;
                reinterpret_cast<float4 *>(part + c)[i] = make_float4(a[0], a[1], a[2], a[3]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (c + i < d) part[c + i] = acc[j * VEC + i];
        }
    }
}

// the same where each slot's rows have a lead of their own, so that a thread's
// channels are not those of its place in another slot: joined by channel
template <int VEC, int NC>
__device__ __forceinline__ void block_part_shifted(const float *acc, int t, int tpr, int lead, int slot, int slots, int d,
                                                   float *part, float *buf) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = (j * tpr + t) * VEC - lead + i;
            if (c >= 0 && c < d) buf[slot * d + c] = acc[j * VEC + i];
        }
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += blockDim.x) {
        float sum = buf[c];
        for (int i = 1; i < slots; ++i) sum += buf[i * d + c];
        part[c] = sum;
    }
}

// ---- the rows of the gated norm: (b, l, h) with h innermost, or, where a
// block stays with one head, (b, l).  Positions are found anew for every row,
// by two multiplications for divisions: a walk that steps offsets along keeps
// twenty registers more, which the backward pass has not (38 against 30 us).
FastDiv fast_div(unsigned by) {
    // n / by = n * ceil(2^(31 + s) / by) >> (31 + s), s = ceil(log2 by), for n < 2^31
    FastDiv f{by, 0, 0};
    while ((1u << f.shift) < by) ++f.shift;
    f.factor = (unsigned)(((1ull << (31 + f.shift)) + by - 1) / by);
    return f;
}
__device__ __forceinline__ unsigned divide(unsigned n, const FastDiv &f) {
    return f.by == 1 ? n : __umulhi(n, f.factor) >> (f.shift - 1);
}

// The offsets of a row's first channel in an array of strided rows (b*sb +
// h*sh + l*sl), in one of tokens (ld apart) and in one of tokens without gaps.
// Where all fit 31 bits (p.small), in 32-bit arithmetic.
struct GateOffsets {
    long long strided, tokens, packed;
};
// row `row` of the kernel's; `head`: the block's, or 0
__device__ __forceinline__ GateOffsets gate_offsets(const NormGateParams &p, long long row, int head, long long sb,
                                                    long long sh, long long sl, long long ld) {
    GateOffsets r;
    if (p.small) {
        const unsigned n = (unsigned)row, token = divide(n, p.heads), h = head + (n - token * p.heads.by);
        const unsigned b = divide(token, p.tokens), l = token - b * p.tokens.by;
        r.strided = b * (unsigned)sb + h * (unsigned)sh + l * (unsigned)sl;
        r.tokens = token * (unsigned)ld + h * (unsigned)p.d;
        r.packed = (token * (unsigned)p.H + h) * (unsigned)p.d;
    } else {
        const long long token = row / p.heads.by, h = head + (row - token * p.heads.by);
        const long long b = token / p.L, l = token - b * p.L;
        r.strided = b * sb + h * sh + l * sl;
        r.tokens = token * ld + h * p.d;
        r.packed = (token * p.H + h) * p.d;
    }
    return r;
}

// Blocks per SM that the registers have to leave room for: threads up to 256,
// 512 (16 channels each) and 1024 (rows beyond 8192).
constexpr int fwd_blocks(int mt, int each = 8) { return mt > 256 ? 1 : each == 8 ? 4 : each == 16 ? 3 : 2; }
constexpr int bwd_blocks(int mt, int vec = 8, int each = 8) { return mt > 256 ? 1 : vec == 1 || each == 16 ? 2 : 3; }

template <typename T, int VEC, int NC, int MT, bool GATE>
__global__ void __launch_bounds__(MT, fwd_blocks(MT, VEC * NC)) norm_gate_kernel(NormGateParams p, int tpr, int parts) {
    constexpr int E = VEC * NC;
    using Rows = Ahead<T, VEC, NC, GATE ? 2 : 1, MT, fwd_blocks(MT, VEC * NC)>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[2][32][2];
    const int t = threadIdx.x % tpr, slot = threadIdx.x / tpr, slots = blockDim.x / tpr, d = p.d;
    Rows rows(smem, t, tpr, d);
    const int head = p.per_head ? blockIdx.x / parts : 0;
    const long long first = (long long)(blockIdx.x % parts) * slots, step = (long long)parts * slots;
    const long long end = (long long)p.B * p.L * (p.per_head ? 1 : p.H);
    long long ahead = first + slot;
    auto fetch = [&](int stage) {
        const bool ok = ahead < end;
        const GateOffsets at = gate_offsets(p, ok ? ahead : 0, head, p.o_sb, p.o_sh, p.o_sl, p.ldg);
        rows.fetch(stage, 0, static_cast<const T *>(p.o) + at.strided, ok);
        if constexpr (GATE) rows.fetch(stage, 1, static_cast<const T *>(p.gate) + at.tokens, ok);
        rows.close();
        ahead += step;
    };
    for (int i = 0; i < Rows::kAhead; ++i) fetch(i);
    float wt[E];
    load_weights<VEC, NC>(wt, p.weight ? p.weight + (long long)head * d : nullptr, t, tpr, d);
    int parity = 0, stage = 0;
    for (long long base = first; base < end; base += step, parity ^= 1) {
        fetch(Rows::last(stage));
        rows.wait();
        float ov[E], sum[1] = {0.f};
        rows.get(stage, 0, ov);
#pragma unroll
        for (int e = 0; e < E; ++e) sum[0] = fmaf(ov[e], ov[e], sum[0]);
        row_sum<1>(sum, tpr, slot, red, parity);
        const float rstd = inv_rms(sum[0] / d, p.eps);
#pragma unroll
        for (int e = 0; e < E; ++e) ov[e] *= rstd * wt[e];
        if constexpr (GATE) {
            float zv[E];
            rows.get(stage, 1, zv);
#pragma unroll
            for (int e = 0; e < E; ++e) ov[e] *= zv[e] * sigmoid(zv[e]);
        }
        const long long row = base + slot;
        if (row < end) rows.store(static_cast<T *>(p.out) + (p.per_head ? row * p.H + head : row) * d, ov);
        stage = Rows::next(stage);
    }
}

template <typename T, int VEC, int NC, int MT, bool GATE>
__global__ void __launch_bounds__(MT, bwd_blocks(MT, VEC, VEC * NC)) norm_gate_bwd_kernel(NormGateParams p, int tpr, int parts) {
    constexpr int E = VEC * NC;
    using Rows = Ahead<T, VEC, NC, GATE ? 3 : 2, MT, bwd_blocks(MT, VEC, VEC * NC)>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[2][32][2];
    const int t = threadIdx.x % tpr, slot = threadIdx.x / tpr, slots = blockDim.x / tpr, d = p.d;
    Rows rows(smem, t, tpr, d);
    const int head = p.per_head ? blockIdx.x / parts : 0;
    const long long first = (long long)(blockIdx.x % parts) * slots, step = (long long)parts * slots;
    const long long end = (long long)p.B * p.L * (p.per_head ? 1 : p.H);
    long long ahead = first + slot;
    auto fetch = [&](int stage) {
        const bool ok = ahead < end;
        const GateOffsets at = gate_offsets(p, ok ? ahead : 0, head, p.o_sb, p.o_sh, p.o_sl, p.ldg);
        rows.fetch(stage, 0, static_cast<const T *>(p.o) + at.strided, ok);
        rows.fetch(stage, 1, static_cast<const T *>(p.dout) + at.packed, ok);
        if constexpr (GATE) rows.fetch(stage, 2, static_cast<const T *>(p.gate) + at.tokens, ok);
        rows.close();
        ahead += step;
    };
    for (int i = 0; i < Rows::kAhead; ++i) fetch(i);
    float wt[E], dw[E];
    load_weights<VEC, NC>(wt, p.weight ? p.weight + (long long)head * d : nullptr, t, tpr, d);
#pragma unroll
    for (int e = 0; e < E; ++e) dw[e] = 0.f;
    const float inv_d = 1.f / d;
    int parity = 0, stage = 0;
    for (long long base = first; base < end; base += step, parity ^= 1) {
        fetch(Rows::last(stage));
        rows.wait();
        float ov[E], zv[E], gv[E], sum[2] = {0.f, 0.f};
        rows.get(stage, 0, ov);
        rows.get(stage, 1, gv);
        if constexpr (GATE) rows.get(stage, 2, zv);
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
        row_sum<2>(sum, tpr, slot, red, parity);
        const float rstd = inv_rms(sum[0] * inv_d, p.eps);
        const float m = sum[1] * inv_d * rstd * rstd;  // mean(e w n) r
#pragma unroll
        for (int e = 0; e < E; ++e) {
            dw[e] = fmaf(gv[e], ov[e] * rstd, dw[e]);
            ov[e] = fmaf(-ov[e], m, gv[e] * wt[e]) * rstd;
            if constexpr (GATE) zv[e] *= rstd;
        }
        const long long row = base + slot;
        if (row < end) {
            const GateOffsets at = gate_offsets(p, row, head, p.do_sb, p.do_sh, p.do_sl, p.lddg);
            rows.store(static_cast<T *>(p.d_o) + at.strided, ov);
            if constexpr (GATE) rows.store(static_cast<T *>(p.dgate) + at.tokens, zv);
        }
        stage = Rows::next(stage);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Rows::wait_all();  // the block's sums take the copies' place
    if (p.dweight)
        block_part<VEC, NC>(dw, t, tpr, slot, slots, d,
                            p.ws + ((long long)(blockIdx.x % parts) * (p.per_head ? p.H : 1) + head) * d,
                            reinterpret_cast<float *>(smem));
}

template <typename T, int VEC, int NC, int MT, bool ADD, bool SHIFT>
__global__ void __launch_bounds__(MT, fwd_blocks(MT, VEC * NC)) residual_norm_kernel(ResidualNormParams p, int tpr) {
    constexpr int E = VEC * NC;
    using Rows = Ahead<T, VEC, NC, ADD ? 2 : 1, MT, fwd_blocks(MT, VEC * NC), SHIFT>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[2][32][2];
    const int t = threadIdx.x % tpr, slot = threadIdx.x / tpr, slots = blockDim.x / tpr, d = p.D;
    const long long step = (long long)gridDim.x * slots;
    long long row = (long long)blockIdx.x * slots + slot, ahead = row;
    Rows rows(smem, t, tpr, d, (int)((unsigned)row * (unsigned)d) & (VEC - 1));
    auto fetch = [&](int stage) {
        const bool ok = ahead < p.R;
        const long long at = ok ? ahead * d : 0;
        rows.fetch(stage, 0, static_cast<const T *>(p.r) + at, ok);
        if constexpr (ADD) rows.fetch(stage, 1, static_cast<const T *>(p.y) + at, ok);
        rows.close();
        ahead += step;
    };
    for (int i = 0; i < Rows::kAhead; ++i) fetch(i);
    float wt[E], sc[E];
    load_weights<VEC, NC>(wt, p.weight, t, tpr, d, rows.lead);
    if constexpr (ADD) load_weights<VEC, NC>(sc, p.scale, t, tpr, d, rows.lead);
    int parity = 0, stage = 0;
    for (long long base = (long long)blockIdx.x * slots; base < p.R; base += step, parity ^= 1) {
        fetch(Rows::last(stage));
        rows.wait();
        float v[E], sum[1] = {0.f};
        rows.get(stage, 0, v);
        if constexpr (ADD) {
            float y[E];
            rows.get(stage, 1, y);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = fmaf(sc[e], y[e], v[e]);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) sum[0] = fmaf(v[e], v[e], sum[0]);
        row_sum<1>(sum, tpr, slot, red, parity);
        const float rstd = inv_rms(sum[0] / d, p.eps);
        const bool ok = row < p.R;
        if (ok && p.r_out) rows.store(static_cast<T *>(p.r_out) + row * d, v);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= rstd * wt[e];
        if (ok) rows.store(static_cast<T *>(p.h) + row * d, v);
        row += step;
        stage = Rows::next(stage);
    }
}

template <typename T, int VEC, int NC, int MT, bool ADD, bool SHIFT>
__global__ void __launch_bounds__(MT, bwd_blocks(MT, VEC, VEC * NC)) residual_norm_bwd_kernel(ResidualNormParams p, int tpr) {
    constexpr int E = VEC * NC;
    using Rows = Ahead<T, VEC, NC, ADD ? 4 : 3, MT, bwd_blocks(MT, VEC, VEC * NC), SHIFT>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[2][32][2];
    const int t = threadIdx.x % tpr, slot = threadIdx.x / tpr, slots = blockDim.x / tpr, d = p.D;
    const long long step = (long long)gridDim.x * slots;
    long long row = (long long)blockIdx.x * slots + slot, ahead = row;
    Rows rows(smem, t, tpr, d, (int)((unsigned)row * (unsigned)d) & (VEC - 1));
    const bool stream = p.dr_out != nullptr;
    auto fetch = [&](int stage) {
        const bool ok = ahead < p.R;
        const long long at = ok ? ahead * d : 0;
        rows.fetch(stage, 0, static_cast<const T *>(p.r) + at, ok);
        rows.fetch(stage, 1, static_cast<const T *>(p.dh) + at, ok);
        rows.fetch(stage, 2, static_cast<const T *>(stream ? p.dr_out : p.dh) + at, ok && stream);
        if constexpr (ADD) rows.fetch(stage, 3, static_cast<const T *>(p.y) + at, ok);
        rows.close();
        ahead += step;
    };
    for (int i = 0; i < Rows::kAhead; ++i) fetch(i);
    float wt[E], sc[E], dw[E], ds[E];
    // Eight channels of aligned rows: one by one.  The loop behind loads of four
    // takes longer (65536x2048 in bf16 284 against 275 us; 9x2048 4.5 against 4.9).
    constexpr bool kFours = SHIFT || E > 8;
    load_weights<VEC, NC, kFours>(wt, p.weight, t, tpr, d, rows.lead);
    load_weights<VEC, NC, kFours>(sc, p.scale, t, tpr, d, rows.lead);
#pragma unroll
    for (int e = 0; e < E; ++e) dw[e] = ds[e] = 0.f;
    const float inv_d = 1.f / d;
    int parity = 0, stage = 0;
    for (long long base = (long long)blockIdx.x * slots; base < p.R; base += step, parity ^= 1) {
        fetch(Rows::last(stage));
        rows.wait();
        float v[E], x[E], sum[2] = {0.f, 0.f};
        rows.get(stage, 0, v);
        rows.get(stage, 1, x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            sum[0] = fmaf(v[e], v[e], sum[0]);
            sum[1] = fmaf(x[e] * wt[e], v[e], sum[1]);
        }
        row_sum<2>(sum, tpr, slot, red, parity);
        const float rstd = inv_rms(sum[0] * inv_d, p.eps);
        const float m = sum[1] * inv_d * rstd * rstd;  // mean(e n) r
        rows.get(stage, 0, v);  // widened again: held across the sums they would take registers
        rows.get(stage, 1, x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            dw[e] = fmaf(x[e], v[e] * rstd, dw[e]);
            x[e] = fmaf(-v[e], m, x[e] * wt[e]) * rstd;
        }
        rows.get(stage, 2, v);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] += v[e];
        if constexpr (ADD) {
            rows.get(stage, 3, v);
#pragma unroll
            for (int e = 0; e < E; ++e) ds[e] = fmaf(x[e], v[e], ds[e]);
        }
        if (row < p.R) {
            rows.store(static_cast<T *>(p.dr) + row * d, x);
            if (p.dy) {
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] *= sc[e];
                rows.store(static_cast<T *>(p.dy) + row * d, x);
            }
        }
        row += step;
        stage = Rows::next(stage);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Rows::wait_all();
    float *buf = reinterpret_cast<float *>(smem);
    auto join = [&](float *acc, long long at) {
        if constexpr (SHIFT)
            block_part_shifted<VEC, NC>(acc, t, tpr, rows.lead, slot, slots, d, p.ws + at * d, buf);
        else
            block_part<VEC, NC>(acc, t, tpr, slot, slots, d, p.ws + at * d, buf);
    };
    if (p.dweight) join(dw, blockIdx.x);
    if constexpr (ADD)
        if (p.dscale) join(ds, (long long)gridDim.x + blockIdx.x);
}

// out[c] = sum over i of part[i*n + c]: 32 channels per block, kSegments runs
// of partial sums side by side, joined in order; blockIdx.y takes the second
// set of partial sums (behind the first) and its output.  Latency is all there
// is to it: 8 segments took 12 us for 444 partial sums, 32 take 4.  Launched
// early (programmatic serialisation), it waits here for the sums.
__global__ void __launch_bounds__(32 * kSegments) sum_parts_kernel(const float *part, int parts, long long n,
                                                                   float *out0, float *out1) {
    __shared__ float seg[kSegments][33];
    float *out = blockIdx.y ? out1 : out0;
    const int lane = threadIdx.x % 32, s = threadIdx.x / 32;
    const long long c = (long long)blockIdx.x * 32 + lane;
    const float *at = part + (long long)blockIdx.y * parts * n;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float acc = 0.f;
    if (out && c < n)
#pragma unroll 16
        for (int i = s; i < parts; i += kSegments) acc += at[i * n + c];
    seg[s][lane] = acc;
    __syncthreads();
    // warp s joins the segments of channel s
    static_assert(kSegments == 32, "a warp per channel");
    float v = group_sum<32>(seg[lane][s]);
    const long long mine = (long long)blockIdx.x * 32 + s;
    if (lane == 0 && out && mine < n) out[mine] = v;
}

// ---- launches

// How a row of d channels is laid on threads.  Backward: 8 channels a thread
// (16 beyond 2048, and in the gated norm, which has one weight to accumulate:
// 30 against 27 us at 8x12x2048x64), so that the accumulators of the weights'
// gradients stay in registers.  Forward there are none: 16 beyond 64 channels, which halves what
// a row costs beside its channels, and up to 1024 channels a row stays inside a
// warp, which needs no barrier, with up to 32 (not in single elements, whose
// loads are held in registers one by one).
//
// A block's warps go round the SM's four schedulers, so five warps take a block
// as long as eight: what a row costs is the channels that its turns could
// carry, `carried`.  Beyond 1024 channels a forward row that fills less than
// four fifths of that takes 24 or 32 channels a thread where they carry less,
// if there are rows for blocks on every SM (16384 rows of bf16: 27 against 35 us
// of 1112 channels, 36 against 42 of 1536, 92 against 136 of 4097; of 6000, which
// fill theirs, 16 channels take 128 and 24 take 146).  fp32, with twice the
// bytes to a channel, gains up to 2048 only (54 against 60 us of 1111; 202 against
// 177 of 4097).
enum Kind { kForward, kGateBackward, kResidualBackward };
struct Layout {
    int each, tpr, threads, slots;
    Layout(int d, Kind kind, int vec = 1, long long rows = 0) {
        int channels = d > 2048 || (kind == kGateBackward && vec > 1 && d > 32) ? 16 : 8;
        if (kind == kForward && vec > 1 && d > 64 && d <= 1024) channels = d <= 256 ? 16 : (d + 255) / 256 * 8;
        lay(d, channels);
        if (kind != kForward || vec == 1 || d <= 1024 || d > (vec == 4 ? 2048 : 8192) || d * 5 >= carried() * 4) return;
        const Layout first = *this;
        Layout best = first;
        for (int more = 24; more <= 32; more += 8) {
            lay(d, more);
            if (threads <= 256 && rows >= (long long)slots * kSms &&
                (carried() < best.carried() || (best.each == first.each && carried() == best.carried())))
                best = *this;
        }
        *this = best;
    }
    void lay(int d, int channels) {
        each = channels;
        const int need = (d + each - 1) / each;
        if (need > 32) {
            tpr = (need + 31) / 32 * 32;
        } else {
            tpr = 1;
            while (tpr < need) tpr *= 2;
        }
        slots = tpr >= 256 ? 1 : 256 / tpr;
        threads = tpr * slots;
    }
    int carried() const { return each * ((threads + 127) / 128 * 128) / slots; }
    // blocks for `rows` rows: `per_sm` (of at most 256 threads) on every SM, at
    // least `least` rows each where there are as many
    int blocks(long long rows, int per_sm, int least) const {
        const long long want = (rows + (long long)slots * least - 1) / ((long long)slots * least);
        const int held = 256 * per_sm / threads > 1 ? 256 * per_sm / threads : 1;
        return (int)(want < (long long)kSms * held ? want : (long long)kSms * held);
    }
    int forward_blocks(long long rows) const { return blocks(rows, fwd_blocks(256, each), 1); }
    // `all`: the rows of all heads
    int backward_blocks(long long rows, long long all) const {
        const long long fill = all / ((long long)slots * kSms);  // rows each, one block on every SM
        return blocks(rows, bwd_blocks(256, 8, each), fill >= kMinRows ? kMinRows : fill > 1 ? (int)fill : 1);
    }
};

bool vec_ok(const void *p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool two_ok(const void *p) { return !p || (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// the widest pieces that all of the arrays and strides allow: 16 bytes, two
// bf16, or single elements
template <typename T> int pieces(std::initializer_list<const void *> arrays, std::initializer_list<long long> strides) {
    bool wide = true, two = sizeof(T) == 2;
    for (const void *p : arrays) wide = wide && vec_ok(p), two = two && two_ok(p);
    for (long long s : strides) wide = wide && s % (16 / (int)sizeof(T)) == 0, two = two && s % 2 == 0;
    return wide ? 16 / (int)sizeof(T) : two ? 2 : 1;
}

// go(VEC, NC, threads' limit) for the layout's channels a thread
template <typename T, bool FORWARD, typename F> int with_layout(const Layout &lay, int vec, F go) {
    using std::integral_constant;
    auto sized = [&](auto v) {
        constexpr int V = decltype(v)::value;
        if (lay.threads > 512) return go(v, integral_constant<int, 16 / V>(), integral_constant<int, 1024>());
        if (lay.threads > 256) return go(v, integral_constant<int, 16 / V>(), integral_constant<int, 512>());
        if constexpr (FORWARD && V > 1) {
            if (lay.each == 24) return go(v, integral_constant<int, 24 / V>(), integral_constant<int, 256>());
            if (lay.each == 32) return go(v, integral_constant<int, 32 / V>(), integral_constant<int, 256>());
        }
        if (lay.each == 16) return go(v, integral_constant<int, 16 / V>(), integral_constant<int, 256>());
        return go(v, integral_constant<int, 8 / V>(), integral_constant<int, 256>());
    };
    if (vec == 16 / (int)sizeof(T)) return sized(integral_constant<int, 16 / (int)sizeof(T)>());
    if constexpr (sizeof(T) == 2)
        if (vec == 2) return sized(integral_constant<int, 2>());
    return sized(integral_constant<int, 1>());
}

// shared memory of a block of `threads`: the rows ahead; the block's sums use it later
template <typename T, int VEC, int NC, int A, int MT, int BLOCKS> constexpr size_t ring_bytes(int threads) {
    const size_t ring = (size_t)threads * Ahead<T, VEC, NC, A, MT, BLOCKS>::kBytes, sums = (size_t)threads * VEC * NC * sizeof(float);
    return ring > sums ? ring : sums;
}

// a launch with its dynamic shared memory; `most`, what the kernel's largest
// block takes, is allowed once per kernel and device
template <auto kernel, typename... A>
int launch(unsigned grid, int threads, size_t smem, size_t most, cudaStream_t s, const A &...args) {
    static std::atomic<unsigned> allowed{0};
    int dev = 0;
    if (most > 32 * 1024 && cudaGetDevice(&dev) == cudaSuccess && (dev >= 32 || !(allowed.load() >> dev & 1))) {
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (dev < 32) allowed.fetch_or(1u << dev);
    }
    kernel<<<grid, threads, smem, s>>>(args...);
    return 0;
}

// sum_parts_kernel behind the kernel that writes the sums, its launch overlapping that one's end
int launch_sums(const float *part, int parts, long long n, float *out0, float *out1, cudaStream_t s) {
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)((n + 31) / 32), out1 ? 2 : 1);
    c.blockDim = dim3(32 * kSegments);
    c.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    if (cudaLaunchKernelEx(&c, sum_parts_kernel, part, parts, n, out0, out1) == cudaSuccess) return 0;
    cudaGetLastError();
    return -7;
}

// the blocks of the gated norm, per head where each stays with one
int gate_parts(const Layout &lay, const NormGateParams &p, bool forward) {
    const long long every = (long long)p.B * p.L * p.H;
    auto blocks = [&](long long rows) { return forward ? lay.forward_blocks(rows) : lay.backward_blocks(rows, every); };
    if (!p.per_head) return blocks(every);
    // every head has blocks of its own: share the device's between them
    const int all = blocks((long long)p.B * p.L), share = (blocks(1ll << 60) + p.H - 1) / p.H;
    return all < share ? all : share;
}

// p with its divisions
NormGateParams divided(NormGateParams p) {
    p.heads = fast_div(p.per_head ? 1u : (unsigned)p.H);
    p.tokens = fast_div((unsigned)p.L);
    const long long tokens = (long long)p.B * p.L, most = 1ll << 31;
    auto strided = [&](long long sb, long long sh, long long sl) {
        return (p.B - 1) * sb < most && (p.H - 1) * sh < most && (p.L - 1) * sl < most &&
               (p.B - 1) * sb + (p.H - 1) * sh + (p.L - 1) * sl < most;
    };
    auto rows = [&](long long ld) { return tokens == 1 || (ld < most && tokens * ld < most); };
    p.small = tokens < most / p.H / p.d && rows(p.ldg) && rows(p.lddg) && strided(p.o_sb, p.o_sh, p.o_sl) &&
              strided(p.do_sb, p.do_sh, p.do_sl);
    return p;
}

// the rows of the residual norm: their layout, and whether they are shifted (a
// layout then has room for the lead, and blocks walk rows in steps after which
// the lead repeats)
constexpr int kShiftThreads = 512;
struct ResidualRows {
    int d, vec;
    bool shift;
    Layout lay;
    ResidualRows(int R, int d_, Kind kind, int vec_, bool shift_)
        : d(d_), vec(vec_), shift(shift_), lay(shift_ ? d_ + vec_ - 1 : d_, kind, vec_, R) {}
    int whole(int blocks, int most) const {
        int q = 1;
        while (shift && (long long)q * lay.slots * d % vec) q *= 2;
        const int up = (blocks + q - 1) / q * q;
        return up <= most ? up : most / q * q;
    }
    int forward_blocks(long long rows) const { return whole(lay.forward_blocks(rows), lay.forward_blocks(1ll << 60)); }
    int backward_blocks(long long rows) const {
        return whole(lay.backward_blocks(rows, rows), lay.backward_blocks(1ll << 60, 1ll << 60));
    }
};
template <typename T> ResidualRows residual_rows(int R, int d, Kind kind, std::initializer_list<const void *> arrays) {
    constexpr int wide = 16 / (int)sizeof(T);
    const int vec = pieces<T>(arrays, {d});
    bool shift = vec < wide;
    for (const void *p : arrays) shift = shift && vec_ok(p);
    const ResidualRows shifted(R, d, kind, wide, true);
    return shift && shifted.lay.threads <= kShiftThreads ? shifted : ResidualRows(R, d, kind, vec, false);
}

}  // namespace

size_t norm_gate_bwd_ws_bytes(int, int B, int H, int L, int d) {
    // for any alignment, and weights of either kind
    NormGateParams p{};
    p.B = B; p.H = H; p.L = L;
    size_t most = 0;
    for (int vec = 1; vec <= 2; ++vec)
        for (p.per_head = 0; p.per_head < 2; ++p.per_head) {
            const size_t n = (size_t)gate_parts(Layout(d, kGateBackward, vec), p, false) * (p.per_head ? H : 1) * d;
            most = n > most ? n : most;
        }
    return sizeof(float) * most;
}
size_t residual_norm_bwd_ws_bytes(int, int R, int D) {
    // for any type and alignment
    const int plain = Layout(D, kResidualBackward).backward_blocks(R, R);
    const int four = ResidualRows(R, D, kResidualBackward, 4, true).backward_blocks(R),
              eight = ResidualRows(R, D, kResidualBackward, 8, true).backward_blocks(R);
    return sizeof(float) * 2 * (size_t)std::max(plain, std::max(four, eight)) * D;
}

template <typename T> int launch_norm_gate(const NormGateParams &q, cudaStream_t s) {
    const NormGateParams p = divided(q);
    const int vec = pieces<T>({p.o, p.gate, p.out}, {p.d, p.o_sb, p.o_sh, p.o_sl, p.gate ? p.ldg : 0});
    const Layout lay(p.d, kForward, vec, (long long)p.B * p.L * (p.per_head ? 1 : p.H));
    const int parts = gate_parts(lay, p, true);
    const unsigned grid = (unsigned)parts * (p.per_head ? p.H : 1);
    return with_layout<T, true>(lay, vec, [&](auto v, auto nc, auto mt) {
        constexpr int V = v(), N = nc(), M = mt(), B = fwd_blocks(M, V * N);
        return p.gate ? launch<norm_gate_kernel<T, V, N, M, true>>(grid, lay.threads, ring_bytes<T, V, N, 2, M, B>(lay.threads), ring_bytes<T, V, N, 2, M, B>(M), s, p, lay.tpr, parts)
                      : launch<norm_gate_kernel<T, V, N, M, false>>(grid, lay.threads, ring_bytes<T, V, N, 1, M, B>(lay.threads), ring_bytes<T, V, N, 1, M, B>(M), s, p, lay.tpr, parts);
    });
}

template <typename T> int launch_norm_gate_bwd(const NormGateParams &q, cudaStream_t s) {
    const NormGateParams p = divided(q);
    const int vec = pieces<T>({p.o, p.gate, p.dout, p.d_o, p.dgate},
                              {p.d, p.o_sb, p.o_sh, p.o_sl, p.do_sb, p.do_sh, p.do_sl, p.gate ? p.ldg : 0, p.gate ? p.lddg : 0});
    const Layout lay(p.d, kGateBackward, vec);
    const int parts = gate_parts(lay, p, false);
    const unsigned grid = (unsigned)parts * (p.per_head ? p.H : 1);
    with_layout<T, false>(lay, vec, [&](auto v, auto nc, auto mt) {
        constexpr int V = v(), N = nc(), M = mt(), B = bwd_blocks(M, V, V * N);
        return p.gate ? launch<norm_gate_bwd_kernel<T, V, N, M, true>>(grid, lay.threads, ring_bytes<T, V, N, 3, M, B>(lay.threads), ring_bytes<T, V, N, 3, M, B>(M), s, p, lay.tpr, parts)
                      : launch<norm_gate_bwd_kernel<T, V, N, M, false>>(grid, lay.threads, ring_bytes<T, V, N, 2, M, B>(lay.threads), ring_bytes<T, V, N, 2, M, B>(M), s, p, lay.tpr, parts);
    });
    if (!p.dweight) return 0;
    const long long n = (long long)p.d * (p.per_head ? p.H : 1);
    return launch_sums(p.ws, parts, n, p.dweight, nullptr, s);
}

template <typename T> int launch_residual_norm(const ResidualNormParams &p, cudaStream_t s) {
    const auto rows = residual_rows<T>(p.R, p.D, kForward, {p.r, p.y, p.r_out, p.h});
    const unsigned grid = (unsigned)rows.forward_blocks(p.R);
    return with_layout<T, true>(rows.lay, rows.vec, [&](auto v, auto nc, auto mt) {
        constexpr int V = v(), N = nc(), M = mt(), B = fwd_blocks(M, V * N);
        auto go = [&](auto add, auto shift) {
            constexpr int A = add() ? 2 : 1;
            return launch<residual_norm_kernel<T, V, N, M, add(), shift()>>(
                grid, rows.lay.threads, ring_bytes<T, V, N, A, M, B>(rows.lay.threads), ring_bytes<T, V, N, A, M, B>(M), s, p, rows.lay.tpr);
        };
        if constexpr (V == 16 / (int)sizeof(T) && M <= kShiftThreads)
            if (rows.shift) return p.y ? go(std::true_type(), std::true_type()) : go(std::false_type(), std::true_type());
        return p.y ? go(std::true_type(), std::false_type()) : go(std::false_type(), std::false_type());
    });
}

template <typename T> int launch_residual_norm_bwd(const ResidualNormParams &p, cudaStream_t s) {
    const auto rows = residual_rows<T>(p.R, p.D, kResidualBackward, {p.r, p.y, p.dh, p.dr_out, p.dr, p.dy});
    const unsigned grid = (unsigned)rows.backward_blocks(p.R);
    with_layout<T, false>(rows.lay, rows.vec, [&](auto v, auto nc, auto mt) {
        constexpr int V = v(), N = nc(), M = mt(), B = bwd_blocks(M, V, V * N);
        auto go = [&](auto add, auto shift) {
            constexpr int A = add() ? 4 : 3;
            return launch<residual_norm_bwd_kernel<T, V, N, M, add(), shift()>>(
                grid, rows.lay.threads, ring_bytes<T, V, N, A, M, B>(rows.lay.threads), ring_bytes<T, V, N, A, M, B>(M), s, p, rows.lay.tpr);
        };
        if constexpr (V == 16 / (int)sizeof(T) && M <= kShiftThreads)
            if (rows.shift) return p.y ? go(std::true_type(), std::true_type()) : go(std::false_type(), std::true_type());
        return p.y ? go(std::true_type(), std::false_type()) : go(std::false_type(), std::false_type());
    });
    if (p.dweight || p.dscale) return launch_sums(p.ws, (int)grid, p.D, p.dweight, p.dscale, s);
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
