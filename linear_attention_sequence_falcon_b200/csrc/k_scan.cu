// k_scan.cu -- the gated linear recurrence (falcon_scan), its backward pass
// and its single-token step:
//   a_t = 1/(1+exp(-f_t)),  c_t = 1 - a_t,
//   h_t = (reset_t ? 0 : a_t h_{t-1}) + c_t x_t.
//
// A run of tokens is an affine map of the state in front of it, h -> A h + B,
// and two maps one behind the other are one: (A2 A1, A2 B1 + B2).  So the
// tokens of one (sequence, group of channels) are cut into runs of kRun
// tokens, one thread per run and pair of channels; a thread block takes a
// tile of runs, and a cluster of blocks takes neighbouring tiles at once and
// walks the sequence.  Each thread forms its run's map from registers; the
// maps of the tile are joined through shared memory, those of the cluster's
// tiles through distributed shared memory: every block sends its tile's map to
// all of its cluster (st.async, counted by the receiver's mbarrier, so that no
// store to global memory has to be waited for, as a cluster barrier's release
// would); then the thread applies its map to the state that enters its run and
// writes.  Every input is read once.  The order of all joins is fixed by the
// token's position alone, so results do not depend on the cluster's size.
//
// The backward pass walks the other way with the same products A:
//   g_t = dout_t + y_t,  y_{t-1} = (reset_t ? 0 : a_t g_t),
// whose run map is y -> A y + sum_t (a_first ... a_t) dout_t, formed in the
// same forward loop; the states come from the marks that the forward left
// every kScanBlock tokens.
//
// A map that contains a reset ignores what comes before, infinities and NaN
// included: its A is -0.0 (no product of gates is), and it is applied by
// selection, not by multiplication.
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "params_layer.h"
#include "tc_sm100.cuh"

namespace falcon {

namespace {

constexpr int kThreads = 256;  // 8 warps per block
constexpr int kMaxCluster = 8;
constexpr uint64_t kGiveUpNs = 2000000000ull;  // a wait for the cluster's maps

__device__ unsigned int g_scan_wait_timeouts;

// ---- pairs of fp32 in one instruction
__device__ __forceinline__ unsigned long long bits(float2 v) { return *reinterpret_cast<unsigned long long *>(&v); }
__device__ __forceinline__ float2 pair(unsigned long long v) { return *reinterpret_cast<float2 *>(&v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return pair(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
    return pair(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
    return pair(d);
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// a = sigmoid(f), c = 1 - a, each to full relative accuracy, without a branch
// on f's sign: e = exp(-f), a = 1/(1+e), c = e a.  The exponent is held at
// 115 (f = -79.7: a is 2e-35 from there on), so that e a stays finite.
__device__ __forceinline__ void gates(float2 f, float2 &a, float2 &c) {
    const float2 z = mul2(f, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    const float2 e = make_float2(ex2(min_nan(z.x, 115.f)), ex2(min_nan(z.y, 115.f)));
    const float2 s = add2(e, make_float2(1.f, 1.f));
    a = make_float2(rcp(s.x), rcp(s.y));
    c = mul2(e, a);
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
        const float x = in0 ? to_f32(p[0]) : fill, y = in1 ? to_f32(p[gap]) : fill;
        r.set(x, y);
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

// The exchange of the tiles' maps inside a cluster.  Step s uses half s & 1 of
// `maps`: a block sends step s + 2 only after every block's map of step s + 1
// has come, which each sends after its reads of step s.
template <int LPR> struct Cluster {
    float4 maps[2][kMaxCluster][LPR];
    uint64_t bar[2];
    int gave_up;

    __device__ __forceinline__ void begin(int cs) {
        if (threadIdx.x == 0) {
            gave_up = 0;
            tc::mbar_init(&bar[0], 1);
            tc::mbar_init(&bar[1], 1);
            tc::fence_mbar_init();
        }
        if (cs > 1) {  // no block writes to another before that runs and its barriers stand
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
    __device__ __forceinline__ void end(int cs) {
        if (cs == 1) return;
        __syncthreads();
        if (threadIdx.x == 0 && gave_up) atomicAdd(&g_scan_wait_timeouts, 1u);
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    }
};

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

// The place of a thread: LPR lanes, a pair of channels each, per run of RUN
// tokens; 32/LPR runs per warp.
template <int LPR, int RUN> struct Place {
    static constexpr int kChannels = 2 * LPR;
    static constexpr int kRuns = kThreads / LPR;      // per tile
    static constexpr int kTile = kRuns * RUN;         // tokens
    static constexpr int kMark = kScanBlock / RUN;    // runs between two marks
};

constexpr int kRun = 8;  // tokens of a run

// One array's rows as a thread meets them.  Inside a tile that is whole (all
// tokens, all channels) an element is at a 32-bit offset from the tile's first
// byte: the strides are at most 2^21 elements, a tile is at most 512 tokens.
template <typename T, bool V, int RUN> struct Rows {
    const char *base;   // the sequence's first token, channel 0
    long long ld;       // bytes from token to token
    uint32_t off;       // this thread's first token and channel, in a tile
    __device__ __forceinline__ Rows(const void *p, long long elements, long long stride, int u, int ch)
        : base(static_cast<const char *>(p) + elements * (long long)sizeof(T)),
          ld(stride * (long long)sizeof(T)),
          off((uint32_t)(u * RUN) * (uint32_t)ld + (uint32_t)(ch * (int)sizeof(T))) {}
    template <bool WHOLE>
    __device__ __forceinline__ Raw<T> load(long long tile0, int i, int gap, bool in0, bool in1, float fill) const {
        const T *p = reinterpret_cast<const T *>(base + tile0 * ld + (off + (uint32_t)i * (uint32_t)ld));
        if constexpr (WHOLE) return load_pair<T, V>(p, gap, true, true, fill);
        else return load_pair<T, V>(p, gap, in0, in1, fill);
    }
    template <bool WHOLE>
    __device__ __forceinline__ void store(long long tile0, int i, int gap, bool in0, bool in1, float2 v) const {
        T *p = reinterpret_cast<T *>(const_cast<char *>(base) + tile0 * ld + (off + (uint32_t)i * (uint32_t)ld));
        if constexpr (WHOLE) store_pair<T, V>(p, gap, true, true, v);
        else store_pair<T, V>(p, gap, in0, in1, v);
    }
};

template <typename T, bool V, int LPR, bool R>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) scan_kernel(ScanParams p) {
    constexpr int RUN = kRun;
    using G = Place<LPR, RUN>;
    __shared__ float4 agg[2][kThreads];
    __shared__ Cluster<LPR> cl;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, u = threadIdx.x / LPR;
    const int cs = (int)cluster_size(), rank = (int)cluster_rank();
    cl.begin(cs);
    const int groups = (p.D + G::kChannels - 1) / G::kChannels;
    const int unit_id = blockIdx.x / cs, n = unit_id / groups;
    const int ch0 = (unit_id % groups) * G::kChannels, ch = ch0 + (V ? 2 * l : l);
    constexpr int gap = LPR;
    const bool in0 = ch < p.D, in1 = V ? in0 : ch + gap < p.D, wide = ch0 + G::kChannels <= p.D;
    const int nblk = (p.L + kScanBlock - 1) / kScanBlock;
    const int tiles = (p.L + G::kTile - 1) / G::kTile, steps = (tiles + cs - 1) / cs;
    const Rows<T, V, RUN> x(p.x, (long long)n * p.L * p.ldx, p.ldx, u, ch);
    const Rows<T, V, RUN> f(p.f, (long long)n * p.L * p.ldf, p.ldf, u, ch);
    const Rows<T, V, RUN> out(p.out, (long long)n * p.L * p.D, p.D, u, ch);
    const float *init = p.init_state ? p.init_state + (long long)n * p.D + ch : nullptr;

    float2 carry = make_float2(init && in0 ? init[0] : 0.f, init && in1 ? init[V ? 1 : gap] : 0.f);
    Raw<T> rx[RUN], rf[RUN];
    uint32_t rr = 0;
    auto fetch = [&](int step) {
        if (step >= steps) return;
        const int tile0 = (step * cs + rank) * G::kTile, t0 = tile0 + u * RUN;
        if constexpr (R) rr = reset_bits<LPR, RUN>(p.reset, (long long)n * p.L + t0, p.L - t0, lane);
        if (wide && tile0 + G::kTile <= p.L) {
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                rx[i] = x.template load<true>(tile0, i, gap, true, true, 0.f);
                rf[i] = f.template load<true>(tile0, i, gap, true, true, 0.f);
            }
        } else {
#pragma unroll
            for (int i = 0; i < RUN; ++i) {  // tokens behind the end keep the state: f = +inf
                const bool in = t0 + i < p.L;
                rx[i] = x.template load<false>(tile0, i, gap, in && in0, in && in1, 0.f);
                rf[i] = f.template load<false>(tile0, i, gap, in && in0, in && in1, __int_as_float(0x7f800000));
            }
        }
    };
    fetch(0);
    for (int step = 0; step < steps; ++step) {
        const int tile0 = (step * cs + rank) * G::kTile, t0 = tile0 + u * RUN, par = step & 1;
        if (cs > 1 && threadIdx.x == 0) tc::mbar_arrive_expect_tx(&cl.bar[par], cs * LPR * sizeof(float4));
        // the run from a zero state: pa = product of the gates up to here, hl = the state
        float2 pa[RUN], hl[RUN];
        const uint32_t cut = rr;
        const int first = R && cut ? __ffs(cut) - 1 : RUN;
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            float2 a, c;
            gates(rf[i].f(), a, c);
            const float2 b = mul2(c, rx[i].f());
            const bool r = R && (cut >> i & 1);
            hl[i] = i == 0 || r ? b : fma2(a, hl[i - 1], b);
            pa[i] = i == 0 ? a : mul2(a, pa[i - 1]);
            if (R && i >= first) pa[i] = make_float2(-0.f, -0.f);
        }
        agg[par][threadIdx.x] = as4({pa[RUN - 1], hl[RUN - 1]});
        fetch(step + 1);
        __syncthreads();
        if (cs > 1 && cl.gave_up) break;
        // the map in front of this run, and, for those who pass it on, the tile's
        Map before = unit();
        for (int i = 0; i < u; ++i) before = join<R>(load_map(&agg[par][i * LPR + l]), before);
        float2 h = carry;
        if (cs == 1 || warp < cs) {
            Map all = before;
            for (int i = u; i < G::kRuns; ++i) all = join<R>(load_map(&agg[par][i * LPR + l]), all);
            if (cs == 1) carry = apply<R>(all, h);
            else if (lane < LPR) send(&cl.maps[par][rank][l], &cl.bar[par], warp, as4(all));
        }
        if (cs > 1) {
            cl.wait(step);
            float2 mine = h;
            for (int i = 0; i < cs; ++i) {
                if (i == rank) mine = h;
                h = apply<R>(load_map(&cl.maps[par][i][l]), h);
            }
            carry = h;
            h = mine;
        }
        h = apply<R>(before, h);
        if (p.marks && u % G::kMark == 0 && t0 < p.L)
            store_pair<float, false>(p.marks + ((long long)n * nblk + t0 / kScanBlock) * p.D + ch, V ? 1 : gap, in0,
                                     in1, h);
        if (!p.out) continue;
        if (wide && tile0 + G::kTile <= p.L) {
#pragma unroll
            for (int i = 0; i < RUN; ++i)
                out.template store<true>(tile0, i, gap, true, true, R && i >= first ? hl[i] : fma2(pa[i], h, hl[i]));
        } else {
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                const bool in = t0 + i < p.L;
                out.template store<false>(tile0, i, gap, in && in0, in && in1,
                                          R && i >= first ? hl[i] : fma2(pa[i], h, hl[i]));
            }
        }
    }
    if (p.final_state && rank == 0 && threadIdx.x < LPR)
        store_pair<float, false>(p.final_state + (long long)n * p.D + ch, V ? 1 : gap, in0, in1, carry);
    cl.end(cs);
}

template <typename T, bool V, int LPR, bool R>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(ScanBwdParams p) {
    constexpr int RUN = kRun;
    using G = Place<LPR, RUN>;
    constexpr bool kAhead = sizeof(T) == 2;  // the next tile's loads before this one's joins (fp32: no registers)
    __shared__ float4 agg[2][kThreads];      // product of the gates, y's map
    __shared__ float2 fwd[2][kThreads];      // the state's B
    __shared__ Cluster<LPR> cl;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, u = threadIdx.x / LPR;
    const int cs = (int)cluster_size(), rank = (int)cluster_rank();
    cl.begin(cs);
    const int groups = (p.D + G::kChannels - 1) / G::kChannels;
    const int unit_id = blockIdx.x / cs, n = unit_id / groups;
    const int ch0 = (unit_id % groups) * G::kChannels, ch = ch0 + (V ? 2 * l : l);
    constexpr int gap = LPR;
    const bool in0 = ch < p.D, in1 = V ? in0 : ch + gap < p.D, wide = ch0 + G::kChannels <= p.D;
    const int nblk = (p.L + kScanBlock - 1) / kScanBlock;
    const int tiles = (p.L + G::kTile - 1) / G::kTile, steps = (tiles + cs - 1) / cs;
    const Rows<T, V, RUN> x(p.x, (long long)n * p.L * p.ldx, p.ldx, u, ch);
    const Rows<T, V, RUN> f(p.f, (long long)n * p.L * p.ldf, p.ldf, u, ch);
    const Rows<T, V, RUN> dout(p.dout, (long long)n * p.L * p.D, p.D, u, ch);
    const Rows<T, V, RUN> dx(p.dx, (long long)n * p.L * p.lddx, p.lddx, u, ch);
    const Rows<T, V, RUN> df(p.df, (long long)n * p.L * p.lddf, p.lddf, u, ch);
    const float *ds = p.dstate ? p.dstate + (long long)n * p.D + ch : nullptr;

    float2 carry = make_float2(ds && in0 ? ds[0] : 0.f, ds && in1 ? ds[V ? 1 : gap] : 0.f);
    Raw<T> rx[RUN], rf[RUN], rd[RUN];
    float2 rm = make_float2(0.f, 0.f);
    uint32_t rr = 0;
    auto fetch = [&](int step) {  // steps from the last tokens to the first
        if (step < 0) return;
        const int tile0 = (step * cs + rank) * G::kTile, t0 = tile0 + u * RUN;
        if constexpr (R) rr = reset_bits<LPR, RUN>(p.reset, (long long)n * p.L + t0, p.L - t0, lane);
        const Raw<float> m = load_pair<float, false>(
            p.marks + ((long long)n * nblk + t0 / kScanBlock) * p.D + ch, V ? 1 : gap, t0 < p.L && in0,
            t0 < p.L && in1, 0.f);
        rm = m.v;
        if (wide && tile0 + G::kTile <= p.L) {
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                rx[i] = x.template load<true>(tile0, i, gap, true, true, 0.f);
                rf[i] = f.template load<true>(tile0, i, gap, true, true, 0.f);
                rd[i] = dout.template load<true>(tile0, i, gap, true, true, 0.f);
            }
        } else {
#pragma unroll
            for (int i = 0; i < RUN; ++i) {  // tokens behind the end hand y on: f = +inf, dout = 0
                const bool in = t0 + i < p.L;
                rx[i] = x.template load<false>(tile0, i, gap, in && in0, in && in1, 0.f);
                rf[i] = f.template load<false>(tile0, i, gap, in && in0, in && in1, __int_as_float(0x7f800000));
                rd[i] = dout.template load<false>(tile0, i, gap, in && in0, in && in1, 0.f);
            }
        }
    };
    if constexpr (kAhead) fetch(steps - 1);
    for (int step = steps - 1; step >= 0; --step) {
        const int turn = steps - 1 - step, par = turn & 1;
        const int tile0 = (step * cs + rank) * G::kTile, t0 = tile0 + u * RUN;
        if (cs > 1 && threadIdx.x == 0) tc::mbar_arrive_expect_tx(&cl.bar[par], cs * LPR * sizeof(float4));
        if constexpr (!kAhead) fetch(step);
        const uint32_t cut = rr;
        const int first = R && cut ? __ffs(cut) - 1 : RUN;
        const float2 mark = rm;
        float2 a[RUN], c[RUN], q[RUN];  // q: c x, later a c (h - x)
        Raw<T> dy[RUN];
        float2 pa, hl, yl = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            gates(rf[i].f(), a[i], c[i]);
            q[i] = mul2(c[i], rx[i].f());
            dy[i] = rd[i];
            const bool r = R && (cut >> i & 1);
            hl = i == 0 || r ? q[i] : fma2(a[i], hl, q[i]);
            pa = i == 0 ? a[i] : mul2(a[i], pa);
            if (R && i >= first) pa = make_float2(-0.f, -0.f);
            else yl = fma2(pa, dy[i].f(), yl);
        }
        agg[par][threadIdx.x] = as4({pa, yl});
        fwd[par][threadIdx.x] = hl;
        if constexpr (kAhead) fetch(step - 1);
        __syncthreads();
        if (cs > 1 && cl.gave_up) break;
        // y's map behind this run, and, for those who pass it on, the tile's
        Map behind = unit();
        for (int i = G::kRuns - 1; i > u; --i) behind = join<R>(load_map(&agg[par][i * LPR + l]), behind);
        float2 y = carry;
        if (cs == 1 || warp < cs) {
            Map all = behind;
            for (int i = u; i >= 0; --i) all = join<R>(load_map(&agg[par][i * LPR + l]), all);
            if (cs == 1) carry = apply<R>(all, y);
            else if (lane < LPR) send(&cl.maps[par][rank][l], &cl.bar[par], warp, as4(all));
        }
        // the state in front of this run, from the mark of its eight
        float2 h = mark;
        for (int i = u & ~(G::kMark - 1); i < u; ++i) {
            const Map m = load_map(&agg[par][i * LPR + l]);
            h = apply<R>({m.a, fwd[par][i * LPR + l]}, h);
        }
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            const bool r = R && (cut >> i & 1);
            const float2 hp = r ? make_float2(0.f, 0.f) : h;
            const float2 b = q[i];
            q[i] = mul2(a[i], fma2(c[i], hp, make_float2(-b.x, -b.y)));
            h = r ? b : fma2(a[i], h, b);
        }
        if (cs > 1) {
            cl.wait(turn);
            float2 mine = y;
            for (int i = cs - 1; i >= 0; --i) {
                if (i == rank) mine = y;
                y = apply<R>(load_map(&cl.maps[par][i][l]), y);
            }
            carry = y;
            y = mine;
        }
        y = apply<R>(behind, y);
        const bool whole = wide && tile0 + G::kTile <= p.L;
#pragma unroll
        for (int i = RUN - 1; i >= 0; --i) {
            const float2 g = add2(dy[i].f(), y);
            if (whole) {
                dx.template store<true>(tile0, i, gap, true, true, mul2(g, c[i]));
                df.template store<true>(tile0, i, gap, true, true, mul2(g, q[i]));
            } else {
                const bool in = t0 + i < p.L;
                dx.template store<false>(tile0, i, gap, in && in0, in && in1, mul2(g, c[i]));
                df.template store<false>(tile0, i, gap, in && in0, in && in1, mul2(g, q[i]));
            }
            y = R && (cut >> i & 1) ? make_float2(0.f, 0.f) : mul2(a[i], g);
        }
    }
    if (p.dinitial && rank == 0 && threadIdx.x < LPR)
        store_pair<float, false>(p.dinitial + (long long)n * p.D + ch, V ? 1 : gap, in0, in1, carry);
    cl.end(cs);
}

template <typename T, bool V>
__global__ void __launch_bounds__(128) scan_step_kernel(ScanStepParams p) {
    const int pairs = (p.D + 1) / 2;
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    if (i >= (long long)p.N * pairs) return;
    const int n = (int)(i / pairs), ch = 2 * (int)(i % pairs);
    const bool in1 = ch + 1 < p.D;
    const long long at = (long long)n * p.D + ch;
    const float2 x = load_pair<T, V>(static_cast<const T *>(p.x) + n * p.ldx + ch, 1, true, in1, 0.f).f();
    const float2 f = load_pair<T, V>(static_cast<const T *>(p.f) + n * p.ldf + ch, 1, true, in1, 0.f).f();
    const float2 s = load_pair<float, V>(p.state + at, 1, true, in1, 0.f).f();
    float2 a, c;
    gates(f, a, c);
    const float2 h = fma2(a, s, mul2(c, x));
    store_pair<float, V>(p.state_out + at, 1, true, in1, h);
    store_pair<T, V>(static_cast<T *>(p.out) + at, 1, true, in1, h);
}

// ---- launches

bool pair_aligned(const void *p, size_t elt, long long ld) {
    return (reinterpret_cast<uintptr_t>(p) & (2 * elt - 1)) == 0 && ld % 2 == 0;
}

// How many clusters of `cs` blocks of a kernel the device holds at once, from
// the occupancy calculator, kept per (kernel, device, cs).
template <typename K> int clusters_held(K kernel, int cs) {
    constexpr int kDevices = 16;
    static std::mutex guard;
    static struct { const void *k; int held[kDevices][kMaxCluster + 1]; } kept[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return 148 * 2 / cs;
    std::lock_guard<std::mutex> lock(guard);
    int *slot = nullptr;
    for (auto &e : kept) {
        if (e.k == nullptr) e.k = reinterpret_cast<const void *>(kernel);
        if (e.k == reinterpret_cast<const void *>(kernel)) { slot = &e.held[dev][cs]; break; }
    }
    if (slot && *slot) return *slot;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(cs * 148);
    c.blockDim = dim3(kThreads);
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cs; at.val.clusterDim.y = 1; at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    int held = 0;
    if (cudaOccupancyMaxActiveClusters(&held, kernel, &c) != cudaSuccess || held < 1) {
        cudaGetLastError();
        held = 1;
    }
    if (slot) *slot = held;
    return held;
}

// The cluster's size: blocks walk steps = tiles/cs tiles each, in as many
// waves as the device needs for all units' clusters; the size with the least
// waves x steps, the smallest of equals (a smaller cluster joins fewer maps).
template <typename K> int pick_cluster(K kernel, long long units, int tiles) {
    int best = 1;
    long long cost = 0;
    for (int cs = 1; cs <= kMaxCluster && cs <= tiles; ++cs) {
        const long long waves = (units + clusters_held(kernel, cs) - 1) / clusters_held(kernel, cs);
        const long long here = waves * ((tiles + cs - 1) / cs);
        if (cs == 1 || here < cost) { best = cs; cost = here; }
    }
    return best;
}

template <typename K, typename P> int launch_units(K kernel, const P &p, long long units, int tiles, cudaStream_t s) {
    const int cs = pick_cluster(kernel, units, tiles);
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(units * cs));
    c.blockDim = dim3(kThreads);
    c.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cs; at.val.clusterDim.y = 1; at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = cs > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&c, kernel, p) == cudaSuccess) return 0;
    cudaGetLastError();
    return -7;
}

// Lanes per run: the fewest that hold the row's pairs, 32 at most.
template <typename F> int with_lanes(int D, F go) {
    if (D <= 8) return go(std::integral_constant<int, 4>());
    if (D <= 16) return go(std::integral_constant<int, 8>());
    if (D <= 32) return go(std::integral_constant<int, 16>());
    return go(std::integral_constant<int, 32>());
}

template <typename F> int with_bools(bool v, bool r, F go) {
    if (v) return r ? go(std::true_type(), std::true_type()) : go(std::true_type(), std::false_type());
    return r ? go(std::false_type(), std::true_type()) : go(std::false_type(), std::false_type());
}

}  // namespace

template <typename T> int launch_scan(const ScanParams &p, cudaStream_t s) {
    const bool v = p.D % 2 == 0 && pair_aligned(p.x, sizeof(T), p.ldx) && pair_aligned(p.f, sizeof(T), p.ldf) &&
                   (!p.out || pair_aligned(p.out, sizeof(T), p.D));
    return with_lanes(p.D, [&](auto lpr) {
        using G = Place<decltype(lpr)::value, kRun>;
        const long long units = (long long)p.N * ((p.D + G::kChannels - 1) / G::kChannels);
        return with_bools(v, p.reset != nullptr, [&](auto vv, auto rr) {
            return launch_units(scan_kernel<T, decltype(vv)::value, decltype(lpr)::value, decltype(rr)::value>, p,
                                units, (p.L + G::kTile - 1) / G::kTile, s);
        });
    });
}

template <typename T> int launch_scan_bwd(const ScanBwdParams &p, cudaStream_t s) {
    const bool v = p.D % 2 == 0 && pair_aligned(p.x, sizeof(T), p.ldx) && pair_aligned(p.f, sizeof(T), p.ldf) &&
                   pair_aligned(p.dout, sizeof(T), p.D) && pair_aligned(p.dx, sizeof(T), p.lddx) &&
                   pair_aligned(p.df, sizeof(T), p.lddf);
    return with_lanes(p.D, [&](auto lpr) {
        using G = Place<decltype(lpr)::value, kRun>;
        const long long units = (long long)p.N * ((p.D + G::kChannels - 1) / G::kChannels);
        return with_bools(v, p.reset != nullptr, [&](auto vv, auto rr) {
            return launch_units(scan_bwd_kernel<T, decltype(vv)::value, decltype(lpr)::value, decltype(rr)::value>, p,
                                units, (p.L + G::kTile - 1) / G::kTile, s);
        });
    });
}

template <typename T> int launch_scan_step(const ScanStepParams &p, cudaStream_t s) {
    const long long pairs = (long long)p.N * ((p.D + 1) / 2);
    const bool v = p.D % 2 == 0 && pair_aligned(p.x, sizeof(T), p.ldx) && pair_aligned(p.f, sizeof(T), p.ldf) &&
                   pair_aligned(p.out, sizeof(T), p.D) && pair_aligned(p.state, 4, 0) && pair_aligned(p.state_out, 4, 0);
    const unsigned blocks = (unsigned)((pairs + 127) / 128);
    if (v) scan_step_kernel<T, true><<<blocks, 128, 0, s>>>(p);
    else scan_step_kernel<T, false><<<blocks, 128, 0, s>>>(p);
    return 0;
}

unsigned int scan_wait_timeouts() {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_scan_wait_timeouts, sizeof(v));
    return v;
}

template int launch_scan<float>(const ScanParams &, cudaStream_t);
template int launch_scan<__nv_bfloat16>(const ScanParams &, cudaStream_t);
template int launch_scan_bwd<float>(const ScanBwdParams &, cudaStream_t);
template int launch_scan_bwd<__nv_bfloat16>(const ScanBwdParams &, cudaStream_t);
template int launch_scan_step<float>(const ScanStepParams &, cudaStream_t);
template int launch_scan_step<__nv_bfloat16>(const ScanStepParams &, cudaStream_t);

}  // namespace falcon
