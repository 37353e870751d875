// scan_parts.cuh -- what the kernels of the gated linear recurrence share
// (k_scan.cu, k_scan_tile.cu): gates, pairs of channels, affine maps of the
// state, their exchange inside a cluster, and the choice of the cluster's size.
#pragma once

#include <type_traits>

#include "cluster_choice.h"
#include "common.cuh"
#include "kernels.h"
#include "params_layer.h"
#include "tc_sm100.cuh"

namespace falcon {
namespace scan {

constexpr uint64_t kGiveUpNs = 2000000000ull;  // a wait for the cluster's maps


// ---- pairs of channels.  One instruction each for the two (f32x2 forms) was
// measured slower here, 187 against 199 us forward at 2x32768x2048: register
// pairs have to be formed for them.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// a = sigmoid(f), c = 1 - a.
//
// Both with relative accuracy, a where it is near 0 too: df and the initial
// state's gradient are proportional to it, and so is the state where x is 0.
// In U = 2^-24 of the value: the exponent's argument is rounded once (with
// log2(e) itself |f| 1.22 U), ex2 is off by 3 U, rcp by 2 U, each sum and
// product by 1 U.
//
// fp32, without a branch on f's sign: e = exp(-f), a = 1/(1+e), c = e a.  The
// exponent is held at 115 (f = -79.7: a is 2e-35 from there on), so that e a
// stays finite; one Newton step takes the reciprocal's last bit, since a
// gradient through a thousand tokens is a product of as many a's (the initial
// state's was off by 6e-7 to 9e-7, with the step by 3e-7).
// bf16: e = exp(f), c = 1/(1+e), and a = 1 - c for f >= 0, where it is off by 3
// U at most and near 1 by its last bit, which counts where products of it are
// long; e c below 0, (1.22 |f| + 7) U off.  (1 - c alone loses a below f = -11
// and is 0 from -17 on.)
template <typename T> __device__ __forceinline__ void gates(float2 f, float2 &a, float2 &c) {
    constexpr float kLog2e = 1.4426950408889634f;
    const float2 one = make_float2(1.f, 1.f);
    if constexpr (sizeof(T) == 2) {
        const float2 z = mul2(f, make_float2(kLog2e, kLog2e)), e = make_float2(ex2(z.x), ex2(z.y)), s = add2(e, one);
        c = make_float2(rcp(s.x), rcp(s.y));
        a = make_float2(e.x < 1.f ? e.x * c.x : 1.f - c.x, e.y < 1.f ? e.y * c.y : 1.f - c.y);
    } else {
        const float2 z = mul2(f, make_float2(-kLog2e, -kLog2e));
        const float2 e = make_float2(ex2(min_nan(z.x, 115.f)), ex2(min_nan(z.y, 115.f)));
        const float2 s = add2(e, one);
        a = make_float2(rcp(s.x), rcp(s.y));
        a = make_float2(fmaf(a.x, fmaf(-s.x, a.x, 1.f), a.x), fmaf(a.y, fmaf(-s.y, a.y, 1.f), a.y));
        c = mul2(e, a);
    }
}

// ---- loads and stores of one thread's two channels (V: next to each other
// and aligned as a pair; otherwise `gap` apart, each by itself)
template <typename T> struct Raw;
template <> struct Raw<float> {
    float2 v;
    __device__ __forceinline__ float2 f() const { return v; }
    __device__ __forceinline__ void set(float x, float y) { v = make_float2(x, y); }
};
template <> struct Raw<__nv_bfloat16> {
    uint32_t v;
    __device__ __forceinline__ float2 f() const {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
    __device__ __forceinline__ void set(float x, float y) {  // values bf16 holds exactly
        v = (__float_as_uint(x) >> 16) | (__float_as_uint(y) & 0xffff0000u);
    }
};

template <typename T, bool V>
__device__ __forceinline__ Raw<T> load_pair(const T *p, int gap, bool in0, bool in1, float fill) {
    Raw<T> r;
    r.set(fill, fill);
    if constexpr (V) {
        if (in0) r.v = *reinterpret_cast<const decltype(r.v) *>(p);
    } else {
        if constexpr (sizeof(T) == 2) {
            const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
            const unsigned short f = __float_as_uint(fill) >> 16, x = in0 ? q[0] : f, y = in1 ? q[gap] : f;
            r.v = (uint32_t)x | (uint32_t)y << 16;
        } else {
            r.v = make_float2(in0 ? p[0] : fill, in1 ? p[gap] : fill);
        }
    }
    return r;
}

template <typename T, bool V>
__device__ __forceinline__ void store_pair(T *p, int gap, bool in0, bool in1, float2 v) {
    if constexpr (V) {
        if (!in0) return;
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<__nv_bfloat162 *>(p) = __float22bfloat162_rn(v);
        else
            *reinterpret_cast<float2 *>(p) = v;
    } else {
        if (in0) p[0] = from_f32<T>(v.x);
        if (in1) p[gap] = from_f32<T>(v.y);
    }
}

// ---- affine maps of a pair of channels
struct Map {
    float2 a, b;
};
__device__ __forceinline__ bool cuts(float a) { return __float_as_uint(a) == 0x80000000u; }
// m applied to h (R: m may contain a reset)
template <bool R> __device__ __forceinline__ float2 apply(const Map &m, float2 h) {
    float2 v = fma2(m.a, h, m.b);
    if constexpr (R) {
        if (cuts(m.a.x)) v.x = m.b.x;
        if (cuts(m.a.y)) v.y = m.b.y;
    }
    return v;
}
// `after` behind `before`, as one map
template <bool R> __device__ __forceinline__ Map join(const Map &after, const Map &before) {
    Map m;
    m.b = apply<R>(after, before.b);
    m.a = mul2(after.a, before.a);
    if constexpr (R) {
        if (cuts(after.a.x)) m.a.x = after.a.x;
        if (cuts(after.a.y)) m.a.y = after.a.y;
    }
    return m;
}
__device__ __forceinline__ Map unit() { return {make_float2(1.f, 1.f), make_float2(0.f, 0.f)}; }

__device__ __forceinline__ Map load_map(const float4 *p) {
    const float4 v = *p;
    return {make_float2(v.x, v.y), make_float2(v.z, v.w)};
}
__device__ __forceinline__ float4 as4(const Map &m) { return make_float4(m.a.x, m.a.y, m.b.x, m.b.y); }

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t remote(const void *p, uint32_t rank) {
    uint32_t to;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(tc::smem_u32(p)), "r"(rank));
    return to;
}
// v to the place of `p`, in the shared memory of `rank`, counted by its `bar`
__device__ __forceinline__ void send(const float4 *p, const uint64_t *bar, uint32_t rank, float4 v) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                     remote(p, rank)),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(remote(bar, rank))
                 : "memory");
}
__device__ __forceinline__ bool wait_parity(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// The exchange of the tiles' maps inside a cluster (shared by the block's
// threads; the maps themselves are in dynamic memory).  Step s uses half s & 1: a block sends step s + 2 only after every block's map of step s + 1
// has come, which each sends after its reads of step s.
template <int LPR> struct Cluster {
    static constexpr size_t kBytes = 2 * LPR * sizeof(float4);  // of the maps [2][cs][LPR], per block of the cluster
    uint64_t bar[2];
    int gave_up;

    __device__ __forceinline__ void begin(int cs) {
        if (threadIdx.x == 0) {
            gave_up = 0;
            tc::mbar_init(&bar[0], 1);
            tc::mbar_init(&bar[1], 1);
            tc::fence_mbar_init();
        }
        if (cs == 1) {
            __syncthreads();
        } else {  // no block writes to another before that runs and its barriers stand
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        }
    }
    // the maps of turn `turn` (0, 1, ...) have come; false: given up
    __device__ __forceinline__ bool wait(int turn) {
        uint64_t *b = &bar[turn & 1];
        const uint32_t parity = (turn >> 1) & 1;
        if (wait_parity(b, parity)) return true;
        const long long t0 = clock64();
        while (!wait_parity(b, parity))
            if (clock64() - t0 > (long long)(2 * kGiveUpNs)) {
                gave_up = 1;
                return false;
            }
        return true;
    }
    // no block leaves while another may still write to it
    __device__ __forceinline__ void end(int cs, unsigned int *timeouts) {
        __syncthreads();
        if (threadIdx.x == 0 && gave_up) atomicAdd(timeouts, 1u);
        if (cs == 1) return;
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    }
};

// The state given has been read (its load is complete) before what follows: the
// state left may be written to the same place, by another thread or block, once
// all of them have passed the barrier or the exchange behind this.
__device__ __forceinline__ void settle(float2 v) { asm volatile("" ::"f"(v.x), "f"(v.y) : "memory"); }

// Which of the run's RUN tokens begin a document, as bits; the LPR lanes of
// a run look at its bytes together.
template <int LPR, int RUN>
__device__ __forceinline__ uint32_t reset_bits(const unsigned char *reset, long long row, int left, int lane) {
    const int l = lane % LPR, base = lane - l;
    uint32_t got = 0;
#pragma unroll
    for (int i = 0; i < RUN; i += LPR) {
        const int t = i + l;
        const bool set = t < RUN && t < left && reset[row + t] != 0;
        got |= ((__ballot_sync(0xffffffffu, set) >> base) & (LPR >= 32 ? 0xffffffffu : (1u << LPR) - 1u)) << i;
    }
    return got & ((1u << RUN) - 1u);
}


// ---- launches

inline bool pair_aligned(const void *p, size_t elt, long long ld) {
    return (reinterpret_cast<uintptr_t>(p) & (2 * elt - 1)) == 0 && ld % 2 == 0;
}

// How many clusters of `cs` blocks of a kernel the device holds at once, from
// the occupancy calculator.  Also lets the kernel have its clusters and its
// dynamic shared memory (of the largest cluster) on that device.
template <typename K> int ask_device(K kernel, int cs, int threads, size_t smem, size_t smem_each) {
    const int most = (int)(smem + kMaxCluster * smem_each);
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(cs * 148);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem + cs * smem_each;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cs; at.val.clusterDim.y = 1; at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    int held = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) == cudaSuccess &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&held, kernel, &c) == cudaSuccess)
        return held;
    cudaGetLastError();
    return kNotAsked;
}

// `smem_each`: shared memory for every block of the cluster, beside `smem`.
template <typename K>
int pick_cluster(K kernel, long long units, int tiles, int threads, size_t smem, size_t smem_each) {
    static ClustersHeld kept;  // of the kernels of this type
    int dev = -1;
    cudaGetDevice(&dev);
    return choose_cluster(units, tiles, [&](int cs) {
        return kept.get(reinterpret_cast<const void *>(kernel), dev, cs,
                        [&] { return ask_device(kernel, cs, threads, smem, smem_each); });
    });
}

template <typename K, typename... P>
int launch_units(K kernel, long long units, int tiles, int threads, size_t smem, size_t smem_each, cudaStream_t s,
                 const P &...p) {
    const int cs = pick_cluster(kernel, units, tiles, threads, smem, smem_each);
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(units * cs));
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem + cs * smem_each;
    c.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cs; at.val.clusterDim.y = 1; at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = cs > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&c, kernel, p...) == cudaSuccess) return 0;
    cudaGetLastError();
    return -7;
}


}  // namespace scan
}  // namespace falcon
