// k_scan_tma.cu -- the gated linear recurrence and its backward pass
// (k_scan.cu has the mathematics) fed by TMA, for rows on 16-byte boundaries.
//
// A tile is 64 tokens by 64 channels: four warps of one run of 16 tokens each,
// a pair of channels per lane.  One thread keeps kStages - 1 tiles in flight
// as tensor copies into a ring in shared memory, so that the loads need
// neither registers nor address arithmetic, and the joins of the maps (one
// per run and tile, and one exchange per step in the cluster) are spread over
// 16 tokens of 2 channels per thread.
#include <cuda.h>

#include "scan_parts.cuh"

namespace falcon {

using namespace scan;

namespace {

constexpr int kRun = 16;            // tokens of a run
constexpr int kWarps = 4;           // runs of a tile
constexpr int kTmaThreads = 32 * kWarps;
constexpr int kTile = kRun * kWarps;
constexpr int kCh = 64;             // channels of a tile
static_assert(kTile == kScanBlock, "a mark in front of every tile");

__device__ unsigned int g_scan_tma_wait_timeouts;

// Tiles of the ring.  Three leave room for one block less per SM: forward
// 160 against 148 us at 2x32768x2048, backward 41 against 31 us at 8x2048x768.
constexpr int kStages = 2;
template <typename T> constexpr int tile_bytes() { return kTile * kCh * (int)sizeof(T); }

struct FwdMaps {
    CUtensorMap x, f;
};
struct BwdMaps {
    CUtensorMap x, f, dout;
};

// The ring: `A` arrays' tiles per stage.
template <typename T, int A> struct Ring {
    static constexpr int S = kStages;
    static constexpr int kStage = A * tile_bytes<T>();
    static constexpr size_t kBytes = (size_t)S * kStage;
    uint8_t *base;
    uint64_t *full;
    int issued;  // turns loaded so far (the loading thread's)

    __device__ __forceinline__ void begin(uint8_t *dynamic, uint64_t *bars) {
        base = dynamic;
        full = bars;
        issued = 0;
        if (threadIdx.x == 0) {
            for (int i = 0; i < S; ++i) tc::mbar_init(&full[i], 1);
            tc::fence_mbar_init();
        }
    }
    // one thread: the tile of turn `turn`
    __device__ __forceinline__ void load(int turn, const CUtensorMap *const (&maps)[A], int ch, int token, int n) {
        const int s = turn % S;
        issued = turn + 1;
        tc::mbar_arrive_expect_tx(&full[s], kStage);
#pragma unroll
        for (int a = 0; a < A; ++a)
            tc::tma_load_3d(tc::smem_u32(base + s * kStage + a * tile_bytes<T>()), maps[a], ch, token, n, &full[s]);
    }
    __device__ __forceinline__ bool wait(int turn) {
        return tc::mbar_wait_timeout(&full[turn % S], (turn / S) & 1, kGiveUpNs);
    }
    // given up: the copies still on their way land before the block's memory goes
    __device__ __forceinline__ void drain() {
        for (int t = issued > S ? issued - S : 0; t < issued; ++t)
            tc::mbar_wait_timeout(&full[t % S], (t / S) & 1, kGiveUpNs / 10);
    }
    // tokens behind the sequence's end (zeros, as the copy fills them) keep the
    // state: f = +inf, each thread at its own channels
    __device__ __forceinline__ void keep_behind(int turn, int a, int at0, int left) const {
        Raw<T> r;
        r.set(__int_as_float(0x7f800000), __int_as_float(0x7f800000));
        for (int i = left < 0 ? 0 : left; i < kRun; ++i)
            *reinterpret_cast<decltype(r.v) *>(base + (turn % S) * kStage + a * tile_bytes<T>() +
                                               (at0 + i * kCh) * (int)sizeof(T)) = r.v;
    }
    // a thread's pair of run token i of array a
    __device__ __forceinline__ Raw<T> get(int turn, int a, int at) const {
        Raw<T> r;
        r.v = *reinterpret_cast<const decltype(r.v) *>(base + (turn % S) * kStage + a * tile_bytes<T>() +
                                                       at * (int)sizeof(T));
        return r;
    }
};

template <typename T, bool R>
__global__ void __launch_bounds__(kTmaThreads, sizeof(T) == 2 ? 4 : 3)
scan_tma_kernel(const __grid_constant__ FwdMaps maps, ScanParams p) {
    extern __shared__ __align__(128) uint8_t dynamic[];
    __shared__ float4 agg[2][kTmaThreads];
    __shared__ Cluster<32> cl;
    __shared__ uint64_t bars[kStages];
    using Tiles = Ring<T, 2>;
    constexpr int S = Tiles::S;
    const int lane = threadIdx.x & 31, u = threadIdx.x >> 5;
    const int cs = (int)cluster_size(), rank = (int)cluster_rank();
    Tiles ring;
    ring.begin(dynamic, bars);
    cl.begin(cs);
    float4 *const maps_of = reinterpret_cast<float4 *>(dynamic + Tiles::kBytes);  // the cluster's tiles' maps, [2][cs][32]
    const int groups = (p.D + kCh - 1) / kCh;
    const int unit_id = blockIdx.x / cs, n = unit_id / groups;
    const int ch0 = (unit_id % groups) * kCh, ch = ch0 + 2 * lane;
    const bool in = ch < p.D;  // D is even
    const int tiles = (p.L + kTile - 1) / kTile, steps = (tiles + cs - 1) / cs;
    const CUtensorMap *const sources[2] = {&maps.x, &maps.f};
    if (threadIdx.x == 0)
        for (int s = 0; s < S && s < steps; ++s) ring.load(s, sources, ch0, (s * cs + rank) * kTile, n);
    float2 carry = make_float2(0.f, 0.f);
    if (p.init_state && in) carry = make_float2(p.init_state[(long long)n * p.D + ch], p.init_state[(long long)n * p.D + ch + 1]);
    uint32_t rr = 0;
    if constexpr (R) rr = reset_bits<32, kRun>(p.reset, (long long)n * p.L + rank * kTile + u * kRun, p.L - rank * kTile - u * kRun, lane);
    for (int step = 0; step < steps; ++step) {
        const int tile0 = (step * cs + rank) * kTile, t0 = tile0 + u * kRun, par = step & 1;
        const int left = p.L - t0;
        if (cs > 1 && threadIdx.x == 0) tc::mbar_arrive_expect_tx(&cl.bar[par], cs * 32 * sizeof(float4));
        const uint32_t cut = rr;
        const int first = R && cut ? __ffs(cut) - 1 : kRun;
        if (!ring.wait(step)) cl.gave_up = 1;
        // the run from a zero state: pa = product of the gates up to here, hl = the state
        float2 pa[kRun], hl[kRun];
        const int at0 = u * kRun * kCh + 2 * lane;
        if (left < kRun) ring.keep_behind(step, 1, at0, left);
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            float2 a, c;
            gates(ring.get(step, 1, at0 + i * kCh).f(), a, c);
            const float2 b = mul2(c, ring.get(step, 0, at0 + i * kCh).f());
            const bool r = R && (cut >> i & 1);
            hl[i] = i == 0 || r ? b : fma2(a, hl[i - 1], b);
            pa[i] = i == 0 ? a : mul2(a, pa[i - 1]);
            if (R && i >= first) pa[i] = make_float2(-0.f, -0.f);
        }
        agg[par][threadIdx.x] = as4({pa[kRun - 1], hl[kRun - 1]});
        if constexpr (R) {
            const int t1 = t0 + cs * kTile;
            rr = reset_bits<32, kRun>(p.reset, (long long)n * p.L + t1, p.L - t1, lane);
        }
        __syncthreads();
        if (cl.gave_up) break;
        if (threadIdx.x == 0 && step + S < steps) ring.load(step + S, sources, ch0, tile0 + S * cs * kTile, n);
        // the map in front of this run, and the tile's
        Map before = unit(), all = load_map(&agg[par][lane]);
#pragma unroll
        for (int i = 1; i < kWarps; ++i) {
            if (i == u) before = all;
            all = join<R>(load_map(&agg[par][i * 32 + lane]), all);
        }
        float2 h = carry;
        if (cs == 1) {
            carry = apply<R>(all, h);
        } else {
            for (int to = u; to < cs; to += kWarps) send(&maps_of[(par * cs + rank) * 32 + lane], &cl.bar[par], to, as4(all));
            cl.wait(step);
            for (int i = 0; i < rank; ++i) h = apply<R>(load_map(&maps_of[(par * cs + i) * 32 + lane]), h);
            carry = h;
            for (int i = rank; i < cs; ++i) carry = apply<R>(load_map(&maps_of[(par * cs + i) * 32 + lane]), carry);
        }
        if (p.marks && u == 0 && left > 0 && in)
            store_pair<float, false>(p.marks + ((long long)n * tiles + step * cs + rank) * p.D + ch, 1, true, true, h);
        h = apply<R>(before, h);
        if (!p.out) continue;
        T *out = static_cast<T *>(p.out) + ((long long)n * p.L + t0) * p.D + ch;
        if (in && left >= kRun) {
#pragma unroll
            for (int i = 0; i < kRun; ++i, out += p.D)
                store_pair<T, true>(out, 1, true, true, R && i >= first ? hl[i] : fma2(pa[i], h, hl[i]));
        } else if (in) {
#pragma unroll
            for (int i = 0; i < kRun; ++i, out += p.D)
                store_pair<T, true>(out, 1, i < left, true, R && i >= first ? hl[i] : fma2(pa[i], h, hl[i]));
        }
    }
    if (p.final_state && rank == 0 && u == 0 && in)
        store_pair<float, false>(p.final_state + (long long)n * p.D + ch, 1, true, true, carry);
    cl.end(cs, &g_scan_tma_wait_timeouts);
    if (cl.gave_up && threadIdx.x == 0) ring.drain();
}

template <typename T, bool R>
__global__ void __launch_bounds__(kTmaThreads, sizeof(T) == 2 ? 3 : 2)
scan_bwd_tma_kernel(const __grid_constant__ BwdMaps maps, ScanBwdParams p) {
    extern __shared__ __align__(128) uint8_t dynamic[];
    __shared__ float4 agg[2][kTmaThreads];  // product of the gates, y's map
    __shared__ float2 fwd[2][kTmaThreads];  // the state's B
    __shared__ Cluster<32> cl;
    __shared__ uint64_t bars[kStages];
    using Tiles = Ring<T, 3>;
    constexpr int S = Tiles::S;
    const int lane = threadIdx.x & 31, u = threadIdx.x >> 5;
    const int cs = (int)cluster_size(), rank = (int)cluster_rank();
    Tiles ring;
    ring.begin(dynamic, bars);
    cl.begin(cs);
    float4 *const maps_of = reinterpret_cast<float4 *>(dynamic + Tiles::kBytes);  // the cluster's tiles' maps, [2][cs][32]
    const int groups = (p.D + kCh - 1) / kCh;
    const int unit_id = blockIdx.x / cs, n = unit_id / groups;
    const int ch0 = (unit_id % groups) * kCh, ch = ch0 + 2 * lane;
    const bool in = ch < p.D;
    const int tiles = (p.L + kTile - 1) / kTile, steps = (tiles + cs - 1) / cs;
    const CUtensorMap *const sources[3] = {&maps.x, &maps.f, &maps.dout};
    // turns count the steps from the last tokens to the first
    if (threadIdx.x == 0)
        for (int s = 0; s < S && s < steps; ++s) ring.load(s, sources, ch0, ((steps - 1 - s) * cs + rank) * kTile, n);
    float2 carry = make_float2(0.f, 0.f);
    if (p.dstate && in) carry = make_float2(p.dstate[(long long)n * p.D + ch], p.dstate[(long long)n * p.D + ch + 1]);
    uint32_t rr = 0;
    float2 rm = make_float2(0.f, 0.f);
    auto ahead = [&](int step) {  // the mark and the resets of a step, a step early
        if (step < 0) return;
        const int tile = step * cs + rank, t0 = tile * kTile + u * kRun;
        if constexpr (R) rr = reset_bits<32, kRun>(p.reset, (long long)n * p.L + t0, p.L - t0, lane);
        if (in && tile < tiles) {
            const float *m = p.marks + ((long long)n * tiles + tile) * p.D + ch;
            rm = make_float2(m[0], m[1]);
        }
    };
    ahead(steps - 1);
    for (int turn = 0; turn < steps; ++turn) {
        const int step = steps - 1 - turn, par = turn & 1;
        const int tile0 = (step * cs + rank) * kTile, t0 = tile0 + u * kRun, left = p.L - t0;
        if (cs > 1 && threadIdx.x == 0) tc::mbar_arrive_expect_tx(&cl.bar[par], cs * 32 * sizeof(float4));
        const uint32_t cut = rr;
        const int first = R && cut ? __ffs(cut) - 1 : kRun;
        float2 h = rm;
        if (!ring.wait(turn)) cl.gave_up = 1;
        float2 a[kRun], c[kRun], q[kRun];  // q: c x, later a c (h - x)
        float2 pa, hl, yl = make_float2(0.f, 0.f);
        const int at0 = u * kRun * kCh + 2 * lane;
        if (left < kRun) ring.keep_behind(turn, 1, at0, left);
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            gates(ring.get(turn, 1, at0 + i * kCh).f(), a[i], c[i]);
            q[i] = mul2(c[i], ring.get(turn, 0, at0 + i * kCh).f());
            const bool r = R && (cut >> i & 1);
            hl = i == 0 || r ? q[i] : fma2(a[i], hl, q[i]);
            pa = i == 0 ? a[i] : mul2(a[i], pa);
            if (R && i >= first) pa = make_float2(-0.f, -0.f);
            else yl = fma2(pa, ring.get(turn, 2, at0 + i * kCh).f(), yl);
        }
        agg[par][threadIdx.x] = as4({pa, yl});
        fwd[par][threadIdx.x] = hl;
        ahead(step - 1);
        __syncthreads();
        if (cl.gave_up) break;
        // every thread has left the tile of the turn before: its place takes the next but S - 1
        if (threadIdx.x == 0 && turn > 0 && turn - 1 + S < steps)
            ring.load(turn - 1 + S, sources, ch0, tile0 - (S - 1) * cs * kTile, n);
        // y's map behind this run, and the tile's
        Map behind = unit(), all = load_map(&agg[par][(kWarps - 1) * 32 + lane]);
#pragma unroll
        for (int i = kWarps - 2; i >= 0; --i) {
            if (i == u) behind = all;
            all = join<R>(load_map(&agg[par][i * 32 + lane]), all);
        }
        float2 y = carry;
        if (cs == 1) carry = apply<R>(all, y);
        else
            for (int to = u; to < cs; to += kWarps) send(&maps_of[(par * cs + rank) * 32 + lane], &cl.bar[par], to, as4(all));
        // the state in front of this run, from the tile's mark
#pragma unroll
        for (int i = 0; i < kWarps - 1; ++i)
            if (i < u) {
                const Map m = load_map(&agg[par][i * 32 + lane]);
                h = apply<R>({m.a, fwd[par][i * 32 + lane]}, h);
            }
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const bool r = R && (cut >> i & 1);
            const float2 hp = r ? make_float2(0.f, 0.f) : h;
            const float2 b = q[i];
            q[i] = mul2(a[i], fma2(c[i], hp, make_float2(-b.x, -b.y)));
            h = r ? b : fma2(a[i], h, b);
        }
        if (cs > 1) {
            cl.wait(turn);
            for (int i = cs - 1; i > rank; --i) y = apply<R>(load_map(&maps_of[(par * cs + i) * 32 + lane]), y);
            carry = y;
            for (int i = rank; i >= 0; --i) carry = apply<R>(load_map(&maps_of[(par * cs + i) * 32 + lane]), carry);
        }
        y = apply<R>(behind, y);
        const long long last = (long long)n * p.L + t0 + kRun - 1;
        T *dx = static_cast<T *>(p.dx) + last * p.lddx + ch, *df = static_cast<T *>(p.df) + last * p.lddf + ch;
        auto finish = [&](auto whole) {
#pragma unroll
            for (int i = kRun - 1; i >= 0; --i, dx -= p.lddx, df -= p.lddf) {
                const float2 g = add2(ring.get(turn, 2, at0 + i * kCh).f(), y);
                if (whole() || i < left) {
                    store_pair<T, true>(dx, 1, true, true, mul2(g, c[i]));
                    store_pair<T, true>(df, 1, true, true, mul2(g, q[i]));
                }
                y = R && (cut >> i & 1) ? make_float2(0.f, 0.f) : mul2(a[i], g);
            }
        };
        if (in && left >= kRun) finish(std::true_type());
        else if (in) finish(std::false_type());
    }
    if (p.dinitial && rank == 0 && u == 0 && in)
        store_pair<float, false>(p.dinitial + (long long)n * p.D + ch, 1, true, true, carry);
    cl.end(cs, &g_scan_tma_wait_timeouts);
    if (cl.gave_up && threadIdx.x == 0) ring.drain();
}

// ---- launches

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
        cudaGetLastError();
    });
    return fn;
}

// [N][L][D] rows `ld` elements apart, tiles of kTile tokens by kCh channels
template <typename T> bool make_map(CUtensorMap *m, const void *base, int N, int L, int D, long long ld) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)L, (cuuint64_t)N};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * sizeof(T), (cuuint64_t)L * ld * sizeof(T)};
    const cuuint32_t box[3] = {kCh, kTile, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
              const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// what a tensor map takes: 16-byte base and strides, strides under 2^40 bytes
template <typename T> bool rows_ok(const void *p, long long ld, int L) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * (int)sizeof(T) % 16 == 0 &&
           (long long)L * ld * (int)sizeof(T) < (1ll << 40);
}

}  // namespace

template <typename T> int launch_scan_tma(const ScanParams &p, cudaStream_t s) {
    if (p.D <= 32 || p.D % 2 || !rows_ok<T>(p.x, p.ldx, p.L) || !rows_ok<T>(p.f, p.ldf, p.L) ||
        (p.out && !pair_aligned(p.out, sizeof(T), p.D)))
        return 1;
    FwdMaps maps;
    if (!make_map<T>(&maps.x, p.x, p.N, p.L, p.D, p.ldx) || !make_map<T>(&maps.f, p.f, p.N, p.L, p.D, p.ldf)) return 1;
    const long long units = (long long)p.N * ((p.D + kCh - 1) / kCh);
    const int tiles = (p.L + kTile - 1) / kTile;
    constexpr size_t smem = Ring<T, 2>::kBytes;
    return p.reset ? launch_units(scan_tma_kernel<T, true>, units, tiles, kTmaThreads, smem, Cluster<32>::kBytes, s, maps, p)
                   : launch_units(scan_tma_kernel<T, false>, units, tiles, kTmaThreads, smem, Cluster<32>::kBytes, s, maps, p);
}

template <typename T> int launch_scan_bwd_tma(const ScanBwdParams &p, cudaStream_t s) {
    if (p.D <= 32 || p.D % 2 || !rows_ok<T>(p.x, p.ldx, p.L) || !rows_ok<T>(p.f, p.ldf, p.L) ||
        !rows_ok<T>(p.dout, p.D, p.L) || !pair_aligned(p.dx, sizeof(T), p.lddx) ||
        !pair_aligned(p.df, sizeof(T), p.lddf))
        return 1;
    BwdMaps maps;
    if (!make_map<T>(&maps.x, p.x, p.N, p.L, p.D, p.ldx) || !make_map<T>(&maps.f, p.f, p.N, p.L, p.D, p.ldf) ||
        !make_map<T>(&maps.dout, p.dout, p.N, p.L, p.D, p.D))
        return 1;
    const long long units = (long long)p.N * ((p.D + kCh - 1) / kCh);
    const int tiles = (p.L + kTile - 1) / kTile;
    constexpr size_t smem = Ring<T, 3>::kBytes;
    return p.reset ? launch_units(scan_bwd_tma_kernel<T, true>, units, tiles, kTmaThreads, smem, Cluster<32>::kBytes, s, maps, p)
                   : launch_units(scan_bwd_tma_kernel<T, false>, units, tiles, kTmaThreads, smem, Cluster<32>::kBytes, s, maps, p);
}

unsigned int scan_tma_wait_timeouts() {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_scan_tma_wait_timeouts, sizeof(v));
    return v;
}

template int launch_scan_tma<float>(const ScanParams &, cudaStream_t);
template int launch_scan_tma<__nv_bfloat16>(const ScanParams &, cudaStream_t);
template int launch_scan_bwd_tma<float>(const ScanBwdParams &, cudaStream_t);
template int launch_scan_bwd_tma<__nv_bfloat16>(const ScanBwdParams &, cudaStream_t);

}  // namespace falcon
