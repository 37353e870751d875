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
#include "scan_parts.cuh"

namespace falcon {

using namespace scan;

namespace {

constexpr int kThreads = 256;  // 8 warps per block

__device__ unsigned int g_scan_wait_timeouts;

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
    extern __shared__ __align__(16) uint8_t dynamic[];
    cl.begin(cs);
    float4 *const maps_of = reinterpret_cast<float4 *>(dynamic);  // the cluster's tiles' maps, [2][cs][LPR]
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
            gates<T>(rf[i].f(), a, c);
            const float2 b = mul2(c, rx[i].f());
            const bool r = R && (cut >> i & 1);
            hl[i] = i == 0 || r ? b : fma2(a, hl[i - 1], b);
            pa[i] = i == 0 ? a : mul2(a, pa[i - 1]);
            if (R && i >= first) pa[i] = make_float2(-0.f, -0.f);
        }
        agg[par][threadIdx.x] = as4({pa[RUN - 1], hl[RUN - 1]});
        fetch(step + 1);
        settle(carry);
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
            else
                for (int to = warp; to < cs && lane < LPR; to += kThreads / 32)
                    send(&maps_of[(par * cs + rank) * LPR + l], &cl.bar[par], to, as4(all));
        }
        if (cs > 1) {
            cl.wait(step);
            for (int i = 0; i < rank; ++i) h = apply<R>(load_map(&maps_of[(par * cs + i) * LPR + l]), h);
            carry = h;
            for (int i = rank; i < cs; ++i) carry = apply<R>(load_map(&maps_of[(par * cs + i) * LPR + l]), carry);
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
    cl.end(cs, &g_scan_wait_timeouts);
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
    extern __shared__ __align__(16) uint8_t dynamic[];
    cl.begin(cs);
    float4 *const maps_of = reinterpret_cast<float4 *>(dynamic);  // the cluster's tiles' maps, [2][cs][LPR]
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
            gates<T>(rf[i].f(), a[i], c[i]);
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
        settle(carry);
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
            else
                for (int to = warp; to < cs && lane < LPR; to += kThreads / 32)
                    send(&maps_of[(par * cs + rank) * LPR + l], &cl.bar[par], to, as4(all));
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
            for (int i = cs - 1; i > rank; --i) y = apply<R>(load_map(&maps_of[(par * cs + i) * LPR + l]), y);
            carry = y;
            for (int i = rank; i >= 0; --i) carry = apply<R>(load_map(&maps_of[(par * cs + i) * LPR + l]), carry);
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
    cl.end(cs, &g_scan_wait_timeouts);
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
    gates<T>(f, a, c);
    const float2 h = fma2(a, s, mul2(c, x));
    store_pair<float, V>(p.state_out + at, 1, true, in1, h);
    store_pair<T, V>(static_cast<T *>(p.out) + at, 1, true, in1, h);
}

// ---- launches

// Lanes per run: the fewest that hold the row's pairs, 32 at most (fp32 alone:
// k_scan_tile.cu has taken every other row of more than 32 channels).
template <typename T, typename F> int with_lanes(int D, F go) {
    if (D <= 8) return go(std::integral_constant<int, 4>());
    if (D <= 16) return go(std::integral_constant<int, 8>());
    if constexpr (sizeof(T) == 4)
        if (D > 32) return go(std::integral_constant<int, 32>());
    return go(std::integral_constant<int, 16>());
}

template <typename F> int with_bools(bool v, bool r, F go) {
    if (v) return r ? go(std::true_type(), std::true_type()) : go(std::true_type(), std::false_type());
    return r ? go(std::false_type(), std::true_type()) : go(std::false_type(), std::false_type());
}

}  // namespace

template <typename T> int launch_scan(const ScanParams &p, cudaStream_t s) {
    const int tile = launch_scan_tile<T>(p, s);
    if (tile != 1) return tile;
    const bool v = p.D % 2 == 0 && pair_aligned(p.x, sizeof(T), p.ldx) && pair_aligned(p.f, sizeof(T), p.ldf) &&
                   (!p.out || pair_aligned(p.out, sizeof(T), p.D));
    return with_lanes<T>(p.D, [&](auto lpr) {
        using G = Place<decltype(lpr)::value, kRun>;
        const long long units = (long long)p.N * ((p.D + G::kChannels - 1) / G::kChannels);
        return with_bools(v, p.reset != nullptr, [&](auto vv, auto rr) {
            return launch_units(scan_kernel<T, decltype(vv)::value, decltype(lpr)::value, decltype(rr)::value>,
                                units, (p.L + G::kTile - 1) / G::kTile, kThreads, 0, Cluster<decltype(lpr)::value>::kBytes, s, p);
        });
    });
}

template <typename T> int launch_scan_bwd(const ScanBwdParams &p, cudaStream_t s) {
    const int tile = launch_scan_bwd_tile<T>(p, s);
    if (tile != 1) return tile;
    const bool v = p.D % 2 == 0 && pair_aligned(p.x, sizeof(T), p.ldx) && pair_aligned(p.f, sizeof(T), p.ldf) &&
                   pair_aligned(p.dout, sizeof(T), p.D) && pair_aligned(p.dx, sizeof(T), p.lddx) &&
                   pair_aligned(p.df, sizeof(T), p.lddf);
    return with_lanes<T>(p.D, [&](auto lpr) {
        using G = Place<decltype(lpr)::value, kRun>;
        const long long units = (long long)p.N * ((p.D + G::kChannels - 1) / G::kChannels);
        return with_bools(v, p.reset != nullptr, [&](auto vv, auto rr) {
            return launch_units(scan_bwd_kernel<T, decltype(vv)::value, decltype(lpr)::value, decltype(rr)::value>,
                                units, (p.L + G::kTile - 1) / G::kTile, kThreads, 0, Cluster<decltype(lpr)::value>::kBytes, s, p);
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
    return v + scan_tile_wait_timeouts();
}

template int launch_scan<float>(const ScanParams &, cudaStream_t);
template int launch_scan<__nv_bfloat16>(const ScanParams &, cudaStream_t);
template int launch_scan_bwd<float>(const ScanBwdParams &, cudaStream_t);
template int launch_scan_bwd<__nv_bfloat16>(const ScanBwdParams &, cudaStream_t);
template int launch_scan_step<float>(const ScanStepParams &, cudaStream_t);
template int launch_scan_step<__nv_bfloat16>(const ScanStepParams &, cudaStream_t);

}  // namespace falcon
