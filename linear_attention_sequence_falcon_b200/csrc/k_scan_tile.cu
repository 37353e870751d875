// k_scan_tile.cu -- the gated linear recurrence and its backward pass
// (k_scan.cu has the mathematics) for more than 32 channels: fp32 rows on
// 16-byte boundaries, bf16 rows on any.
//
// A tile is 64 tokens by 64 channels: four warps of one run of 16 tokens each,
// a pair of channels per lane.  The tiles come through a ring in shared memory,
// so that the loads hold no registers, and the joins of the maps (one per run
// and tile, and one exchange per step in the cluster) are spread over 16 tokens
// of 2 channels per thread.  How they come goes by the alignment of the rows:
//   kTensor   rows on 16-byte boundaries: one thread issues tensor copies
//   kPairs    bf16 rows on 4 bytes, kSingles on 2: every thread loads its own
//             places and stores them into the ring when their turn comes
// Measured for the latter two, forward / backward at 8x2048x514 bf16 (23 / 35
// us so): asynchronous copies of 4 bytes 28 / 39, the loads held in registers
// instead of the ring 26 / 49, runs of 8 tokens held in registers 30 / 44.
// fp32 rows off 16 bytes take the last (k_scan.cu): 20 / 27 against 25 / 38 us
// at 5x1537x515.
#include <cuda.h>

#include "scan_parts.cuh"

namespace falcon {

using namespace scan;

namespace {

constexpr int kRun = 16;            // tokens of a run
constexpr int kWarps = 4;           // runs of a tile
constexpr int kTileThreads = 32 * kWarps;
constexpr int kTile = kRun * kWarps;
constexpr int kCh = 64;             // channels of a tile
static_assert(kTile == kScanBlock, "a mark in front of every tile");

__device__ unsigned int g_scan_tile_wait_timeouts;

// Tiles of the ring.  Three leave room for one block less per SM: forward
// 160 against 148 us at 2x32768x2048, backward 41 against 31 us at 8x2048x768.
constexpr int kStages = 2;

enum Feed { kTensor = 0, kPairs = 1, kSingles = 2 };

struct FwdMaps {
    CUtensorMap x, f;
};
struct BwdMaps {
    CUtensorMap x, f, dout;
};

// One array's rows, for the threads that copy their own places.
struct Source {
    const char *base;   // the sequence's first token, the thread's first channel
    long long ld;       // bytes
};
template <typename T> __device__ __forceinline__ Source source(const void *p, long long ld, int n, int L, int ch) {
    ld *= (int)sizeof(T);
    return {static_cast<const char *>(p) + (long long)n * L * ld + (long long)ch * (int)sizeof(T), ld};
}

// The ring: `A` arrays' tiles per stage.
template <typename T, int A, int FEED> struct Ring {
    static constexpr int S = kStages;
    static constexpr int kTileBytes = kTile * kCh * (int)sizeof(T);
    static constexpr int kStage = A * kTileBytes;
    static constexpr size_t kBytes = (size_t)S * kStage;
    // a thread's two channels: next to each other, or, where they cannot be
    // moved as a pair, 32 apart, so that a warp's single elements are neighbours
    static constexpr bool kPair = FEED != kSingles;
    static constexpr int kGap = kPair ? 1 : 32;
    uint8_t *base;
    uint64_t *full;
    int issued;  // kTensor, the loading thread's: turns loaded so far
    int at0;     // this thread's first place in a tile, in elements

    __device__ __forceinline__ void begin(uint8_t *memory, uint64_t *bars) {
        base = memory;
        full = bars;
        issued = 0;
        at0 = (threadIdx.x >> 5) * kRun * kCh + (threadIdx.x & 31) * (kPair ? 2 : 1);
        if (FEED == kTensor && threadIdx.x == 0) {
            for (int i = 0; i < S; ++i) tc::mbar_init(&full[i], 1);
            tc::fence_mbar_init();
        }
    }
    __device__ __forceinline__ T *place(int turn, int a, int i) const {
        return reinterpret_cast<T *>(base + (turn % S) * kStage + a * kTileBytes) + at0 + i * kCh;
    }
    // kTensor, one thread: the tile of turn `turn`
    __device__ __forceinline__ void load(int turn, const CUtensorMap *const (&maps)[A], int ch, int token, int n) {
        const int s = turn % S;
        issued = turn + 1;
        tc::mbar_arrive_expect_tx(&full[s], kStage);
#pragma unroll
        for (int a = 0; a < A; ++a)
            tc::tma_load_3d(tc::smem_u32(base + s * kStage + a * kTileBytes), maps[a], ch, token, n, &full[s]);
    }
    // otherwise, every thread: its own places, `left` tokens from `token` on;
    // zeros behind the end
    __device__ __forceinline__ void load(int turn, const Source (&from)[A], long long token, int left, bool in0, bool in1) {
        if (left >= kRun && in1) fill<true>(turn, from, token, left, in0, in1);
        else fill<false>(turn, from, token, left, in0, in1);
    }
    template <bool WHOLE>
    __device__ __forceinline__ void fill(int turn, const Source (&from)[A], long long token, int left, bool in0, bool in1) {
#pragma unroll
        for (int a = 0; a < A; ++a) {
            const char *row = from[a].base + token * from[a].ld;
#pragma unroll
            for (int i = 0; i < kRun; ++i, row += from[a].ld) {
                const bool in = WHOLE || i < left;
                T *to = place(turn, a, i);
                if constexpr (kPair) {
                    *reinterpret_cast<uint32_t *>(to) = in && (WHOLE || in0) ? *reinterpret_cast<const uint32_t *>(row) : 0u;
                } else {
                    const T zero = from_f32<T>(0.f), *p = reinterpret_cast<const T *>(row);
                    const T v0 = in && (WHOLE || in0) ? p[0] : zero, v1 = in && (WHOLE || in1) ? p[kGap] : zero;
                    to[0] = v0;
                    to[kGap] = v1;
                }
            }
        }
    }
    // the tile of turn `turn` has come
    __device__ __forceinline__ bool wait(int turn) {
        return FEED != kTensor || tc::mbar_wait_timeout(&full[turn % S], (turn / S) & 1, kGiveUpNs);
    }
    // tokens behind the sequence's end (zeros, as the copies fill them) keep the
    // state: f (array 1) = +inf, each thread at its own channels.  Backward they
    // come first, and a later tile's copy writes the same bytes: the stores are
    // ordered in front of it by the fence here and the barrier before that copy.
    __device__ __forceinline__ void keep_behind(int turn, int left) const {
        const T inf = from_f32<T>(__int_as_float(0x7f800000));
        for (int i = left < 0 ? 0 : left; i < kRun; ++i) place(turn, 1, i)[0] = place(turn, 1, i)[kGap] = inf;
        if constexpr (FEED == kTensor) tc::fence_proxy_async();
    }
    // given up: the copies still on their way land before the block's memory goes
    __device__ __forceinline__ void drain() {
        for (int t = issued > S ? issued - S : 0; t < issued; ++t)
            tc::mbar_wait_timeout(&full[t % S], (t / S) & 1, kGiveUpNs / 10);
    }
    // a thread's pair of run token i of array a
    __device__ __forceinline__ float2 get(int turn, int a, int i) const {
        const T *p = place(turn, a, i);
        if constexpr (kPair) return load_pair<T, true>(p, 1, true, true, 0.f).f();
        else return make_float2(to_f32(p[0]), to_f32(p[kGap]));
    }
};

template <typename T, bool R, int FEED>
__global__ void __launch_bounds__(kTileThreads, sizeof(T) == 2 ? 4 : 3)
scan_tile_kernel(const __grid_constant__ FwdMaps maps, ScanParams p) {
    extern __shared__ __align__(128) uint8_t dynamic[];
    __shared__ float4 agg[2][kTileThreads];
    __shared__ Cluster<32> cl;
    __shared__ uint64_t bars[kStages];
    using Tiles = Ring<T, 2, FEED>;
    constexpr int S = Tiles::S, gap = Tiles::kGap;
    constexpr bool V = Tiles::kPair;
    const int lane = threadIdx.x & 31, u = threadIdx.x >> 5;
    const int cs = (int)cluster_size(), rank = (int)cluster_rank();
    Tiles ring;
    ring.begin(dynamic, bars);
    cl.begin(cs);
    float4 *const maps_of = reinterpret_cast<float4 *>(dynamic + Tiles::kBytes);  // the cluster's tiles' maps, [2][cs][32]
    const int groups = (p.D + kCh - 1) / kCh;
    const int unit_id = blockIdx.x / cs, n = unit_id / groups;
    const int ch0 = (unit_id % groups) * kCh, ch = ch0 + (V ? 2 * lane : lane);
    const bool in0 = ch < p.D, in1 = V ? in0 : ch + gap < p.D;
    const int tiles = (p.L + kTile - 1) / kTile, steps = (tiles + cs - 1) / cs;
    const CUtensorMap *const tensors[2] = {&maps.x, &maps.f};
    const Source rows[2] = {source<T>(p.x, p.ldx, n, p.L, ch), source<T>(p.f, p.ldf, n, p.L, ch)};
    // the tile of step s
    auto load = [&](int s) {
        if constexpr (FEED == kTensor) {
            if (threadIdx.x == 0 && s < steps) ring.load(s, tensors, ch0, (s * cs + rank) * kTile, n);
        } else {
            const int token = (s * cs + rank) * kTile + u * kRun;
            ring.load(s, rows, token, s < steps ? p.L - token : 0, in0, in1);
        }
    };
    if constexpr (FEED == kTensor)
        for (int s = 0; s < S; ++s) load(s);
    float2 carry = make_float2(0.f, 0.f);
    if (p.init_state) carry = load_pair<float, false>(p.init_state + (long long)n * p.D + ch, gap, in0, in1, 0.f).f();
    uint32_t rr = 0;
    if constexpr (R) rr = reset_bits<32, kRun>(p.reset, (long long)n * p.L + rank * kTile + u * kRun, p.L - rank * kTile - u * kRun, lane);
    for (int step = 0; step < steps; ++step) {
        const int tile0 = (step * cs + rank) * kTile, t0 = tile0 + u * kRun, par = step & 1;
        const int left = p.L - t0;
        if (cs > 1 && threadIdx.x == 0) tc::mbar_arrive_expect_tx(&cl.bar[par], cs * 32 * sizeof(float4));
        const uint32_t cut = rr;
        const int first = R && cut ? __ffs(cut) - 1 : kRun;
        if constexpr (FEED != kTensor) load(step);
        if (!ring.wait(step)) cl.gave_up = 1;
        // the run from a zero state: pa = product of the gates up to here, hl = the state
        float2 pa[kRun], hl[kRun];
        if (left < kRun) ring.keep_behind(step, left);
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            float2 a, c;
            gates<T>(ring.get(step, 1, i), a, c);
            const float2 b = mul2(c, ring.get(step, 0, i));
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
        settle(carry);
        __syncthreads();
        if (cl.gave_up) break;
        if constexpr (FEED == kTensor) load(step + S);
        // the map in front of this run, and the tile's
        Map before = unit(), all = load_map(&agg[par][lane]);
        if (u > 0) {  // the branches are the warp's
            before = all;
#pragma unroll
            for (int i = 1; i < kWarps - 1; ++i)
                if (i < u) before = join<R>(load_map(&agg[par][i * 32 + lane]), before);
            all = join<R>({pa[kRun - 1], hl[kRun - 1]}, before);
        }
#pragma unroll
        for (int i = 1; i < kWarps; ++i)
            if (i > u) all = join<R>(load_map(&agg[par][i * 32 + lane]), all);
        float2 h = carry;
        if (cs == 1) {
            carry = apply<R>(all, h);
        } else {
            for (int to = u; to < cs; to += kWarps) send(&maps_of[((par) * cs + rank) * 32 + lane], &cl.bar[par], to, as4(all));
            cl.wait(step);
#pragma unroll 4
            for (int i = 0; i < rank; ++i) h = apply<R>(load_map(&maps_of[((par) * cs + i) * 32 + lane]), h);
            carry = h;
#pragma unroll 4
            for (int i = rank; i < cs; ++i) carry = apply<R>(load_map(&maps_of[((par) * cs + i) * 32 + lane]), carry);
        }
        if (p.marks && u == 0 && left > 0)
            store_pair<float, false>(p.marks + ((long long)n * tiles + step * cs + rank) * p.D + ch, gap, in0, in1, h);
        h = apply<R>(before, h);
        if (!p.out) continue;
        // stores at 32-bit offsets from the tile's first row (strides are at most 2^21)
        char *const out = static_cast<char *>(p.out) + ((long long)n * p.L + tile0) * p.D * (int)sizeof(T);
        const uint32_t pitch = (uint32_t)p.D * (uint32_t)sizeof(T);
        uint32_t at = (uint32_t)(u * kRun) * pitch + (uint32_t)ch * (uint32_t)sizeof(T);
        if (in1 && left >= kRun) {
#pragma unroll
            for (int i = 0; i < kRun; ++i, at += pitch)
                store_pair<T, V>(reinterpret_cast<T *>(out + at), gap, true, true, R && i >= first ? hl[i] : fma2(pa[i], h, hl[i]));
        } else if (in0) {
#pragma unroll
            for (int i = 0; i < kRun; ++i, at += pitch)
                store_pair<T, V>(reinterpret_cast<T *>(out + at), gap, i < left, i < left && in1, R && i >= first ? hl[i] : fma2(pa[i], h, hl[i]));
        }
    }
    if (p.final_state && rank == 0 && u == 0)
        store_pair<float, false>(p.final_state + (long long)n * p.D + ch, gap, in0, in1, carry);
    cl.end(cs, &g_scan_tile_wait_timeouts);
    if (FEED == kTensor && cl.gave_up && threadIdx.x == 0) ring.drain();
}

template <typename T, bool R, int FEED>
__global__ void __launch_bounds__(kTileThreads, sizeof(T) == 2 ? 3 : 2)
scan_bwd_tile_kernel(const __grid_constant__ BwdMaps maps, ScanBwdParams p) {
    extern __shared__ __align__(128) uint8_t dynamic[];
    __shared__ float4 agg[2][kTileThreads];  // product of the gates, y's map
    __shared__ float2 fwd[2][kTileThreads];  // the state's B
    __shared__ Cluster<32> cl;
    __shared__ uint64_t bars[kStages];
    using Tiles = Ring<T, 3, FEED>;
    constexpr int S = Tiles::S, gap = Tiles::kGap;
    constexpr bool V = Tiles::kPair;
    const int lane = threadIdx.x & 31, u = threadIdx.x >> 5;
    const int cs = (int)cluster_size(), rank = (int)cluster_rank();
    Tiles ring;
    ring.begin(dynamic, bars);
    cl.begin(cs);
    float4 *const maps_of = reinterpret_cast<float4 *>(dynamic + Tiles::kBytes);  // the cluster's tiles' maps, [2][cs][32]
    const int groups = (p.D + kCh - 1) / kCh;
    const int unit_id = blockIdx.x / cs, n = unit_id / groups;
    const int ch0 = (unit_id % groups) * kCh, ch = ch0 + (V ? 2 * lane : lane);
    const bool in0 = ch < p.D, in1 = V ? in0 : ch + gap < p.D;
    const int tiles = (p.L + kTile - 1) / kTile, steps = (tiles + cs - 1) / cs;
    const CUtensorMap *const tensors[3] = {&maps.x, &maps.f, &maps.dout};
    const Source rows[3] = {source<T>(p.x, p.ldx, n, p.L, ch), source<T>(p.f, p.ldf, n, p.L, ch),
                            source<T>(p.dout, p.D, n, p.L, ch)};
    // the tile of turn t: turns count the steps from the last tokens to the first
    auto load = [&](int t) {
        const int s = steps - 1 - t;
        if constexpr (FEED == kTensor) {
            if (threadIdx.x == 0 && s >= 0) ring.load(t, tensors, ch0, (s * cs + rank) * kTile, n);
        } else {
            const int token = s < 0 ? 0 : (s * cs + rank) * kTile + u * kRun;
            ring.load(t, rows, token, s < 0 ? 0 : p.L - token, in0, in1);
        }
    };
    if constexpr (FEED == kTensor)
        for (int t = 0; t < S; ++t) load(t);
    float2 carry = make_float2(0.f, 0.f);
    if (p.dstate) carry = load_pair<float, false>(p.dstate + (long long)n * p.D + ch, gap, in0, in1, 0.f).f();
    uint32_t rr = 0;
    float2 rm = make_float2(0.f, 0.f);
    auto ahead = [&](int step) {  // the mark and the resets of a step, a step early
        if (step < 0) return;
        const int tile = step * cs + rank, t0 = tile * kTile + u * kRun;
        if constexpr (R) rr = reset_bits<32, kRun>(p.reset, (long long)n * p.L + t0, p.L - t0, lane);
        if (tile < tiles)
            rm = load_pair<float, false>(p.marks + ((long long)n * tiles + tile) * p.D + ch, gap, in0, in1, 0.f).f();
    };
    ahead(steps - 1);
    for (int turn = 0; turn < steps; ++turn) {
        const int step = steps - 1 - turn, par = turn & 1;
        const int tile0 = (step * cs + rank) * kTile, t0 = tile0 + u * kRun, left = p.L - t0;
        if (cs > 1 && threadIdx.x == 0) tc::mbar_arrive_expect_tx(&cl.bar[par], cs * 32 * sizeof(float4));
        const uint32_t cut = rr;
        const int first = R && cut ? __ffs(cut) - 1 : kRun;
        float2 h = rm;
        if constexpr (FEED != kTensor) load(turn);
        if (!ring.wait(turn)) cl.gave_up = 1;
        float2 a[kRun], c[kRun], q[kRun];  // q: c x, later a c (h - x)
        float2 pa, hl, yl = make_float2(0.f, 0.f);
        if (left < kRun) ring.keep_behind(turn, left);
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            gates<T>(ring.get(turn, 1, i), a[i], c[i]);
            q[i] = mul2(c[i], ring.get(turn, 0, i));
            const bool r = R && (cut >> i & 1);
            hl = i == 0 || r ? q[i] : fma2(a[i], hl, q[i]);
            pa = i == 0 ? a[i] : mul2(a[i], pa);
            if (R && i >= first) pa = make_float2(-0.f, -0.f);
            else yl = fma2(pa, ring.get(turn, 2, i), yl);
        }
        agg[par][threadIdx.x] = as4({pa, yl});
        fwd[par][threadIdx.x] = hl;
        ahead(step - 1);
        settle(carry);
        __syncthreads();
        if (cl.gave_up) break;
        // every thread has left the tile of the turn before: its place takes the next but S - 1
        if constexpr (FEED == kTensor)
            if (turn > 0) load(turn - 1 + S);
        // y's map behind this run, and the tile's
        Map behind = unit(), all = load_map(&agg[par][(kWarps - 1) * 32 + lane]);
        if (u < kWarps - 1) {  // the branches are the warp's
            behind = all;
#pragma unroll
            for (int i = kWarps - 2; i > 0; --i)
                if (i > u) behind = join<R>(load_map(&agg[par][i * 32 + lane]), behind);
            all = join<R>({pa, yl}, behind);
        }
#pragma unroll
        for (int i = kWarps - 2; i >= 0; --i)
            if (i < u) all = join<R>(load_map(&agg[par][i * 32 + lane]), all);
        float2 y = carry;
        if (cs == 1) carry = apply<R>(all, y);
        else
            for (int to = u; to < cs; to += kWarps) send(&maps_of[((par) * cs + rank) * 32 + lane], &cl.bar[par], to, as4(all));
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
#pragma unroll 4
            for (int i = cs - 1; i > rank; --i) y = apply<R>(load_map(&maps_of[((par) * cs + i) * 32 + lane]), y);
            carry = y;
#pragma unroll 4
            for (int i = rank; i >= 0; --i) carry = apply<R>(load_map(&maps_of[((par) * cs + i) * 32 + lane]), carry);
        }
        y = apply<R>(behind, y);
        const long long row0 = (long long)n * p.L + tile0;
        char *const dx = static_cast<char *>(p.dx) + row0 * p.lddx * (int)sizeof(T);
        char *const df = static_cast<char *>(p.df) + row0 * p.lddf * (int)sizeof(T);
        const uint32_t px = (uint32_t)p.lddx * (uint32_t)sizeof(T), pf = (uint32_t)p.lddf * (uint32_t)sizeof(T);
        const uint32_t last = u * kRun + kRun - 1;
        uint32_t at_x = last * px + (uint32_t)ch * (uint32_t)sizeof(T), at_f = last * pf + (uint32_t)ch * (uint32_t)sizeof(T);
        auto finish = [&](auto whole) {
#pragma unroll
            for (int i = kRun - 1; i >= 0; --i, at_x -= px, at_f -= pf) {
                const float2 g = add2(ring.get(turn, 2, i), y);
                const bool here = whole() || i < left;
                store_pair<T, V>(reinterpret_cast<T *>(dx + at_x), gap, here, here && (whole() || in1), mul2(g, c[i]));
                store_pair<T, V>(reinterpret_cast<T *>(df + at_f), gap, here, here && (whole() || in1), mul2(g, q[i]));
                y = R && (cut >> i & 1) ? make_float2(0.f, 0.f) : mul2(a[i], g);
            }
        };
        if (in1 && left >= kRun) finish(std::true_type());
        else if (in0) finish(std::false_type());
    }
    if (p.dinitial && rank == 0 && u == 0)
        store_pair<float, false>(p.dinitial + (long long)n * p.D + ch, gap, in0, in1, carry);
    cl.end(cs, &g_scan_tile_wait_timeouts);
    if (FEED == kTensor && cl.gave_up && threadIdx.x == 0) ring.drain();
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

// go(reset, feed) for arrays whose pairs of channels are aligned, and that tensor maps take
template <typename T, typename F> int with_feed(bool reset, bool tensors, bool pairs, F go) {
    using std::integral_constant;
    auto fed = [&](auto how) { return reset ? go(std::true_type(), how) : go(std::false_type(), how); };
    if (tensors) return fed(integral_constant<int, kTensor>());
    if constexpr (sizeof(T) == 2)
        return pairs ? fed(integral_constant<int, kPairs>()) : fed(integral_constant<int, kSingles>());
    return 1;
}

}  // namespace

template <typename T> int launch_scan_tile(const ScanParams &p, cudaStream_t s) {
    if (p.D <= 32) return 1;
    const bool pairs = p.D % 2 == 0 && pair_aligned(p.x, sizeof(T), p.ldx) && pair_aligned(p.f, sizeof(T), p.ldf) &&
                       (!p.out || pair_aligned(p.out, sizeof(T), p.D));
    FwdMaps maps{};
    const bool tensors = pairs && rows_ok<T>(p.x, p.ldx, p.L) && rows_ok<T>(p.f, p.ldf, p.L) &&
                         make_map<T>(&maps.x, p.x, p.N, p.L, p.D, p.ldx) && make_map<T>(&maps.f, p.f, p.N, p.L, p.D, p.ldf);
    const long long units = (long long)p.N * ((p.D + kCh - 1) / kCh);
    return with_feed<T>(p.reset != nullptr, tensors, pairs, [&](auto r, auto f) {
        return launch_units(scan_tile_kernel<T, r(), f()>, units, (p.L + kTile - 1) / kTile, kTileThreads,
                            Ring<T, 2, f()>::kBytes, Cluster<32>::kBytes, s, maps, p);
    });
}

template <typename T> int launch_scan_bwd_tile(const ScanBwdParams &p, cudaStream_t s) {
    if (p.D <= 32) return 1;
    const bool pairs = p.D % 2 == 0 && pair_aligned(p.x, sizeof(T), p.ldx) && pair_aligned(p.f, sizeof(T), p.ldf) &&
                       pair_aligned(p.dout, sizeof(T), p.D) && pair_aligned(p.dx, sizeof(T), p.lddx) &&
                       pair_aligned(p.df, sizeof(T), p.lddf);
    BwdMaps maps{};
    const bool tensors = pairs && rows_ok<T>(p.x, p.ldx, p.L) && rows_ok<T>(p.f, p.ldf, p.L) && rows_ok<T>(p.dout, p.D, p.L) &&
                         make_map<T>(&maps.x, p.x, p.N, p.L, p.D, p.ldx) && make_map<T>(&maps.f, p.f, p.N, p.L, p.D, p.ldf) &&
                         make_map<T>(&maps.dout, p.dout, p.N, p.L, p.D, p.D);
    const long long units = (long long)p.N * ((p.D + kCh - 1) / kCh);
    return with_feed<T>(p.reset != nullptr, tensors, pairs, [&](auto r, auto f) {
        return launch_units(scan_bwd_tile_kernel<T, r(), f()>, units, (p.L + kTile - 1) / kTile, kTileThreads,
                            Ring<T, 3, f()>::kBytes, Cluster<32>::kBytes, s, maps, p);
    });
}

unsigned int scan_tile_wait_timeouts() {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_scan_tile_wait_timeouts, sizeof(v));
    return v;
}

template int launch_scan_tile<float>(const ScanParams &, cudaStream_t);
template int launch_scan_tile<__nv_bfloat16>(const ScanParams &, cudaStream_t);
template int launch_scan_bwd_tile<float>(const ScanBwdParams &, cudaStream_t);
template int launch_scan_bwd_tile<__nv_bfloat16>(const ScanBwdParams &, cudaStream_t);

}  // namespace falcon
