// Gated linear recurrence, per channel (declarations and contract in include/wkv.h):
//   f_t = sigma(g_t), i_t = 1 - f_t = sigma(-g_t),   h_t = f_t h_{t-1} + i_t x_t,   y_t = h_t
//
// A span of steps maps the state entering it to the state leaving it by
//   h_out = A h_in + H,   A = prod f_t,   H = the span's state from zero,
// and two adjacent spans compose as (A1 A2, A2 H1 + H2), so the long axis is split.  A warp
// takes LC consecutive steps of 32 V adjacent channels and turns each token's gate and input
// into the sums (A_t, H_t) of its steps so far; once it knows the state entering, every output
// is one multiply-add.  The warps of a block cover a tile of adjacent steps, the blocks of a
// cluster adjacent tiles; a cluster walks its channels' sequence in strides of S tiles and
// carries the state from stride to stride.  Summaries meet in (distributed) shared memory, in a
// fixed order: no workspace, no waiting on other clusters, and the same bits on every run.
// Tiles are staged ahead of their use, by TMA where the rows allow it.  Where short sequences have
// channels enough for every warp, nothing is split: a warp walks its channels' whole sequence.
//
// Bound by HBM: g and x are read once, y written once.  B200, forward (backward) against the
// copy rate of 6549 GB/s: 1x16384x4096 fp32 119 us, 6770 GB/s (220 us, 6100 GB/s); 4x4096x2048
// bf16 39.5 us, 5100 GB/s (78.2 us, 4290 GB/s); 64x1024x768 bf16 53.8 us, 5610 GB/s (93.0 us, 5410
// GB/s); 8x1024x768 fp32 15.5 us, 4870 GB/s (26.1 us, 4820 GB/s).  In bf16 a byte carries twice the
// tokens and the warps issue 19 instructions per token forward, 44 backward, in 52 and 60% of the issue
// slots: two or three warps per scheduler, which wait for fixed latencies in between.
//
// Arithmetic: fp32 whatever the I/O type.  A gate is kept as the smaller of (f, i) with a sign,
// from e = 2^(-|g| log2 e) as e / (1 + e), relatively accurate at both ends.  A step starts from
// whichever of h, x it stays near:
//   i <= 1/2:  h - i (h - x)   where a gate holds for thousands of tokens f rounds to within
//                              2^-24 of 1, and repeating f h would drift by that every step;
//   f <  1/2:  x + f (h - x)   a closing gate leaves no rounding of the old state (f = 0: h = x).
// A span passes the state on in the same way, by the smaller of A and 1 - A (span_gate): the state is
// rounded once per span, and the product A itself only serves the span's own outputs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "wkv_device.cuh"
#include "wkv_gated_internal.h"
#include "wkv_internal.h"
#include "wkv_pipe_common.cuh"
#include "wkv_vec.cuh"

namespace wkvb {
namespace {

constexpr int kMaxCluster = 8;  // portable cluster size

struct ScanArgs {
    int64_t B, T, C;
    int64_t groups;  // channel groups per sequence
    int wt_log;      // log2 of the warps of a block along time (NW unless a shorter tile holds T)
    int16_t drop_sums, drop_tile;  // test hook: the block of this rank withholds its sums, or the fetch of its
                                   // first tile (-1: none)
    const void *g, *x, *gy;
    const float* state_in;   // forward: [B][C] or null
    void* y;                 // forward: y; backward: gx
    void* gg;                // backward
    float* state_out;        // forward: state_out; backward: gstate_in; [B][C] or null
    float* carry;            // [B][saved_states(T)][C]: forward writes (or null), backward reads
    const float* gstate;     // backward: gradient of state_out, [B][C] or null
    uint32_t* dev_err;       // the library's device-wide error word
    uint32_t spin_limit;     // bounded waits
};
// The kernels' tensor maps, 128 bytes each, follow it.  Where they straddle two lines of 128 bytes the bf16
// forward is 4 to 6% slower (64x1024x768 53 -> 56).
static_assert(sizeof(ScanArgs) == 128);

__device__ __forceinline__ int64_t saved_states(int64_t T) { return (T + kGatedCarrySteps - 1) / kGatedCarrySteps; }

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// ---- V (1 or 2) adjacent channels per lane: scalars, or pairs on the packed fp32 instructions ----
template <int V>
struct Lanes;
template <>
struct Lanes<1> {
    using T = float;
    static __device__ __forceinline__ T all(float a) { return a; }
    static __device__ __forceinline__ T make(const float (&a)[1]) { return a[0]; }
    static __device__ __forceinline__ void split(T a, float (&o)[1]) { o[0] = a; }
};
template <>
struct Lanes<2> {
    using T = float2;
    static __device__ __forceinline__ T all(float a) { return make_float2(a, a); }
    static __device__ __forceinline__ T make(const float (&a)[2]) { return make_float2(a[0], a[1]); }
    static __device__ __forceinline__ void split(T a, float (&o)[2]) {
        o[0] = a.x;
        o[1] = a.y;
    }
};
__device__ __forceinline__ float vfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 vfma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float vmul(float a, float b) { return a * b; }
__device__ __forceinline__ float2 vmul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float vsub(float a, float b) { return a - b; }
__device__ __forceinline__ float2 vsub(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.f, -1.f), a); }

// ---- the gate, as one signed number s per token: -i where i = sigma(-g) <= 1/2 ("holds": the
// state is kept more than replaced), +f where f = sigma(g) < 1/2; the sign is set on a zero too ----
__device__ __forceinline__ bool holds(float s) { return __float_as_int(s) < 0; }
__device__ __forceinline__ float with_sign_of_minus(float small, float g) {
    return __uint_as_float(__float_as_uint(small) | (~__float_as_uint(g) & 0x80000000u));
}
__device__ __forceinline__ float gate(float g) {
    const float e = ex2(-fabsf(g) * kLog2e);
    return with_sign_of_minus(e * rcp(1.f + e), g);
}
__device__ __forceinline__ float2 gate(float2 g) {
    const float2 e = make_float2(ex2(-fabsf(g.x) * kLog2e), ex2(-fabsf(g.y) * kLog2e));
    const float2 d = __fadd2_rn(e, make_float2(1.f, 1.f));
    const float2 small = __fmul2_rn(e, make_float2(rcp(d.x), rcp(d.y)));
    return make_float2(with_sign_of_minus(small.x, g.x), with_sign_of_minus(small.y, g.y));
}
__device__ __forceinline__ float pick(float s, float if_holds, float if_not) { return holds(s) ? if_holds : if_not; }
__device__ __forceinline__ float2 pick(float2 s, float2 if_holds, float2 if_not) {
    return make_float2(pick(s.x, if_holds.x, if_not.x), pick(s.y, if_holds.y, if_not.y));
}
__device__ __forceinline__ float neg(float a) { return -a; }
__device__ __forceinline__ float2 neg(float2 a) { return make_float2(-a.x, -a.y); }
// A barrier that needs a loaded value: behind it every thread of the block has its own.  A block sends
// its first summary behind it, and the block that writes a cluster's final state has everyone's
// summaries by then, so it may write over the state they began from.
__device__ __forceinline__ void sync_with(float a) { __syncthreads_or(__float_as_int(a) == -1); }
__device__ __forceinline__ void sync_with(float2 a) { __syncthreads_or((__float_as_int(a.x) & __float_as_int(a.y)) == -1); }
__device__ __forceinline__ float zero(float) { return 0.f; }
__device__ __forceinline__ float2 zero(float2) { return make_float2(0.f, 0.f); }

// f h + i x: h - i (h - x), or x + f (h - x)
template <typename T>
__device__ __forceinline__ T gate_step(T s, T h, T x) { return vfma(s, vsub(h, x), pick(s, h, x)); }
// f a: a - i a, or f a
template <typename T>
__device__ __forceinline__ T gate_decay(T s, T a) { return vfma(s, a, pick(s, a, zero(a))); }
// f a, and -i a: -i a, or f a - a
template <typename T>
__device__ __forceinline__ T gate_split(T s, T a, T& input_neg) {
    const T kept = pick(s, a, zero(a));
    input_neg = vfma(s, a, vsub(kept, a));  // kept - a: 0 or -a, exact
    return vfma(s, a, kept);
}
// A span of steps as a gate: its factor A = prod f in the same signed form, from A and Dn = -(1 - A), the
// sum of -i_t A_{t-1} (one fused multiply-add of s and A per step; right while every step holds, and
// A > 1/2 means that every one did).  The product alone, near 1, rounds the same way in span after span:
// with steady gates of logit 9 to 17 (1x16384x64) the final state was off by up to 7600 units of 2^-24 of
// its scale, and is by at most 30 in this form.  It costs 0 to 4% forward and 0 to 7% backward (8x1024x768
// fp32 15.5 and 26.1 us, as before; 4x4096x2048 bf16 39 and 78 against 39 and 75).  Dn starts below zero, so
// that the sign is there from the start.
constexpr float kNoDecay = -1.17549435e-38f;
__device__ __forceinline__ float span_gate(float A, float Dn) { return A > 0.5f ? Dn : A; }
__device__ __forceinline__ float2 span_gate(float2 A, float2 Dn) {
    return make_float2(span_gate(A.x, Dn.x), span_gate(A.y, Dn.y));
}
__device__ __forceinline__ float span_kept(float s) { return s < 0.f ? 1.f : 0.f; }
__device__ __forceinline__ float2 span_kept(float2 s) { return make_float2(span_kept(s.x), span_kept(s.y)); }
// A h + H: h + (H - D h), the difference first, or A h + H
template <typename T>
__device__ __forceinline__ T span_step(T s, T H, T h) { return vfma(span_kept(s), h, vfma(s, h, H)); }
// A a: a - D a, or A a
template <typename T>
__device__ __forceinline__ T span_decay(T s, T a) { return vfma(span_kept(s), a, vmul(s, a)); }
// -f i = s^2 - |s|
__device__ __forceinline__ float gate_slope_neg(float s) { return fmaf(fabsf(s), fabsf(s), -fabsf(s)); }
__device__ __forceinline__ float2 gate_slope_neg(float2 s) { return make_float2(gate_slope_neg(s.x), gate_slope_neg(s.y)); }

// V adjacent channels of LC rows (`stride` elements apart) as fp32; rows from n on are not read
// and come back as `fill`
template <typename TIO, int V, int LC, bool ALL>
__device__ __forceinline__ void load_rows(const TIO* p, int64_t stride, int n, float fill, typename Lanes<V>::T (&o)[LC]) {
#pragma unroll
    for (int s = 0; s < LC; ++s) {
        float t[V];
        if (ALL || s < n) {
            Vec<TIO, V>::load(p + s * stride, t);
        } else {
#pragma unroll
            for (int q = 0; q < V; ++q) t[q] = fill;
        }
        o[s] = Lanes<V>::make(t);
    }
}

// How tiles reach the lanes: from global memory directly; staged by TMA, one box of the tile's rows
// of 32 V channels per array (rows of a multiple of 16 bytes); or staged by 16-byte asynchronous
// copies of each row's segment from the 16-byte boundary before it (any row), 16 bytes of pitch more
// per row.  A copied row begins at its own shift, so a lane's V channels lie 32 apart there, not
// side by side, and are accessed one by one.
enum How { kDirect, kTma, kCopy };

template <typename TIO, int V, int ROWS, How HOW>
struct Tile {
    static constexpr int kPitch = 32 * V * (int)sizeof(TIO) + (HOW == kCopy ? 16 : 0);
    static constexpr int kBytes = ROWS * kPitch;
};

// Whether the backward stages gy in a ring of its own, with ST + 1 slots: read from there twice, it
// takes no registers between, and the others' slots are free as soon as they are in registers.  Not
// for copies, whose addresses would be formed twice (4x1024x2049 bf16: 46 against 31).
template <typename TIO, How HOW>
constexpr bool stages_gy_apart = HOW == kTma && sizeof(TIO) == 2;

// Waits, with a limit, for the end of a mbarrier's phase, whichever it is; runs out where none is under way.
__device__ __forceinline__ void mbar_drain(uint64_t* bar, uint32_t limit) {
    for (uint32_t parity = 0; parity < 2; ++parity) mbar_wait(bar, parity, limit);
}

// A ring of ST staged tiles, completion on the slot's barrier.  A slot is refilled right after the
// block's barrier behind which every lane has its values in registers: by thread 0 (TMA), or by all
// threads (copies).
template <typename TIO, int V, int ROWS, int THREADS, int ARRAYS, int ST, How HOW>
struct Ring {
    using L = Tile<TIO, V, ROWS, HOW>;
    unsigned char* slots;
    uint64_t* full;
    int64_t c0, b, T, C, bytes;  // first channel and sequence; lengths; bytes of an array

    __device__ __forceinline__ void init() {
        for (int i = 0; i < ST; ++i) mbar_init(&full[i], HOW == kCopy ? THREADS : 1);
    }
    __device__ __forceinline__ bool mine() const { return HOW == kCopy || threadIdx.x == 0; }
    // the tile at step t0 into slot it % ST
    __device__ __forceinline__ void fetch(int it, int64_t t0, const CUtensorMap* const* maps, const void* const* from) {
        const int slot = it % ST;
        unsigned char* to = slots + (size_t)slot * ARRAYS * L::kBytes;
        if constexpr (HOW == kTma) {
            mbar_arrive_expect_tx(&full[slot], ARRAYS * L::kBytes);
#pragma unroll
            for (int k = 0; k < ARRAYS; ++k)
                tma_load_3d(to + k * L::kBytes, maps[k], (int)c0, (int)t0, (int)b, &full[slot]);
        } else {
            constexpr int kChunks = L::kPitch / 16;
            const int64_t first = ((b * T + t0) * C + c0) * (int64_t)sizeof(TIO);
            for (int id = threadIdx.x; id < ROWS * kChunks; id += THREADS) {
                const int r = id / kChunks, k = id % kChunks;
                const int64_t start = first + (int64_t)r * C * (int64_t)sizeof(TIO), at = (start & ~(int64_t)15) + 16 * k;
                // nothing past the sequence, past the segment, or past the array's last byte
                int64_t n = t0 + r < T && at < start + 32 * V * (int64_t)sizeof(TIO) ? bytes - at : 0;
                n = n < 0 ? 0 : n > 16 ? 16 : n;
#pragma unroll
                for (int q = 0; q < ARRAYS; ++q)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                     smem_u32(to + q * L::kBytes + r * L::kPitch + 16 * k)),
                                 "l"(static_cast<const unsigned char*>(from[q]) + (n > 0 ? at : 0)), "r"((uint32_t)n)
                                 : "memory");
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&full[slot])) : "memory");
        }
    }
    __device__ __forceinline__ bool wait(int it, uint32_t limit) {
        uint64_t* b = &full[it % ST];
        const uint32_t p = (it / ST) & 1;
        return mbar_try_wait_hint(b, p, kWaitHintNs) || mbar_wait(b, p, limit);
    }
    // every copy under way has landed, or its wait runs out
    __device__ __forceinline__ void drain(uint32_t limit) {
        if (HOW == kCopy) asm volatile("cp.async.wait_all;" ::: "memory");
        for (int i = 0; i < ST; ++i) mbar_drain(&full[i], limit);
    }
    // this lane's channels of row r of array k; `element`: the row's first element within the
    // arrays, modulo 2^32
    __device__ __forceinline__ typename Lanes<V>::T get(int it, int k, int r, uint32_t element) const {
        const unsigned char* row = slots + (size_t)(it % ST * ARRAYS + k) * L::kBytes + r * L::kPitch;
        float t[V];
        if constexpr (HOW == kCopy) {
            const TIO* p = reinterpret_cast<const TIO*>(row + (element * (uint32_t)sizeof(TIO) & 15u)) + (threadIdx.x & 31);
#pragma unroll
            for (int q = 0; q < V; ++q) t[q] = io<TIO>::load(p + 32 * q);
        } else {
            Vec<TIO, V>::load(reinterpret_cast<const TIO*>(row) + (threadIdx.x & 31) * V, t);
        }
        return Lanes<V>::make(t);
    }
};

// The blocks' summaries of one stride, in every block of the cluster: each block sends its own
// to all (st.async: the data and its arrival on the receiver's barrier travel together, so no
// fence has to wait for the outputs still being written).  Two buffers: a block sends stride
// it + 2 only after it has everyone's stride it + 1, and those were sent after their senders
// had read stride it.
template <typename P>
struct Exchange {
    P (*sum)[kMaxCluster][32];
    uint64_t* bar;

    __device__ __forceinline__ void init() {
        mbar_init(&bar[0], 1);
        mbar_init(&bar[1], 1);
    }
    __device__ __forceinline__ void expect(int it, uint32_t S) {
        mbar_arrive_expect_tx(&bar[it & 1], S * 32 * (uint32_t)sizeof(P));
    }
    __device__ __forceinline__ void send(int it, uint32_t S, uint32_t rank, int lane, const P& p) {
        const uint32_t at = smem_u32(&sum[it & 1][rank][lane]), on = smem_u32(&bar[it & 1]);
        for (uint32_t k = 0; k < S; ++k) {
            uint32_t rat, ron;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rat) : "r"(at), "r"(k));
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ron) : "r"(on), "r"(k));
            send_to(rat, ron, p);
        }
    }
    static __device__ __forceinline__ void send_to(uint32_t at, uint32_t on, const float2& p) {
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at),
                     "f"(p.x), "f"(p.y), "r"(on)
                     : "memory");
    }
    static __device__ __forceinline__ void send_to(uint32_t at, uint32_t on, const float4& p) {
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at),
                     "f"(p.x), "f"(p.y), "f"(p.z), "f"(p.w), "r"(on)
                     : "memory");
    }
    __device__ __forceinline__ bool wait(int it, uint32_t limit) {
        return mbar_wait(&bar[it & 1], (it >> 1) & 1, limit);
    }
    // what the others have sent has landed, or the waits run out
    __device__ __forceinline__ void drain(uint32_t limit) {
        mbar_drain(&bar[0], limit);
        mbar_drain(&bar[1], limit);
    }
};

// (A as a signed gate, H) of a span, V channels, as one vector
template <int V>
struct Span;
template <>
struct Span<1> {
    using P = float2;
    static __device__ __forceinline__ P pack(float s, float H) { return make_float2(s, H); }
    static __device__ __forceinline__ float gate(const P& p) { return p.x; }
    static __device__ __forceinline__ float H(const P& p) { return p.y; }
};
template <>
struct Span<2> {
    using P = float4;
    static __device__ __forceinline__ P pack(float2 s, float2 H) { return make_float4(s.x, s.y, H.x, H.y); }
    static __device__ __forceinline__ float2 gate(const P& p) { return make_float2(p.x, p.y); }
    static __device__ __forceinline__ float2 H(const P& p) { return make_float2(p.z, p.w); }
};

// What both directions share: where a lane's channels and steps lie, the hand-over of the state.
template <int V, int LC, int NW, How HOW>
struct Block {
    using T = typename Lanes<V>::T;
    using P = typename Span<V>::P;
    static constexpr bool kStaged = HOW != kDirect;
    // A direct block's few spans hold the whole sequence: plain products, no summaries to pass on.
    static __device__ __forceinline__ T seal(T A, T Dn) { return kStaged ? span_gate(A, Dn) : A; }
    static __device__ __forceinline__ T pass(T s, T H, T h) { return kStaged ? span_step(s, H, h) : vfma(s, h, H); }
    static constexpr int kApart = HOW == kCopy ? 32 : 1;  // from one of a lane's channels to the next
    const ScanArgs& a;
    int lane, warp, WT, wt, W, cl;
    uint32_t S, rank;
    int64_t b, c, tile, tiles;
    bool live, whole;  // this lane's channels exist; so do all of the block's

    __device__ __forceinline__ Block(const ScanArgs& args) : a(args) {
        lane = threadIdx.x & 31;
        warp = threadIdx.x >> 5;
        WT = kStaged ? NW : 1 << a.wt_log;
        wt = kStaged ? warp : warp & (WT - 1);
        const int wc = kStaged ? 0 : warp >> a.wt_log;
        W = kStaged ? 32 * V : (NW >> a.wt_log) * 32 * V;
        cl = HOW == kCopy ? lane : (wc * 32 + lane) * V;
        S = cluster_size();
        rank = cluster_rank();
        const int64_t unit = blockIdx.x / S;
        b = unit / a.groups;
        c = (unit % a.groups) * W + cl;
        live = c < a.C;
        whole = c - cl + W <= a.C;
        tile = (int64_t)WT * LC;
        tiles = (a.T + tile - 1) / tile;
    }
    __device__ __forceinline__ T load_state(const float* p, int64_t row) const {
        float t[V];
#pragma unroll
        for (int q = 0; q < V; ++q) t[q] = 0.f;
        if (p && kApart == 1 && live) Vec<float, V>::load(p + row * a.C + c, t);
        if (p && kApart != 1)
#pragma unroll
            for (int q = 0; q < V; ++q)
                if (c + q * kApart < a.C) t[q] = p[row * a.C + c + q * kApart];
        return Lanes<V>::make(t);
    }
    // `all`: every channel of the block exists
    template <typename TO>
    __device__ __forceinline__ void store(TO* p, T v, bool all) const {
        float t[V];
        Lanes<V>::split(v, t);
        if (kApart == 1) {
            if (all || live) Vec<TO, V>::store(p, t);
        } else {
#pragma unroll
            for (int q = 0; q < V; ++q)
                if (all || c + q * kApart < a.C) io<TO>::store(p + q * kApart, t[q]);
        }
    }
    __device__ __forceinline__ void store_state(float* p, int64_t row, T v) const {
        if (p) store(p + row * a.C + c, v, false);
    }
    // Polls of this thread's bounded waits; 0 once one has run out.  It then fetches, expects and sends
    // nothing: no slot is filled and no phase of a mbarrier begun while the last is under way, since each is
    // begun by a thread that has seen the last one end.  Threads that then miss it run out in turn, once
    // each, the walk goes on to its end without waiting, and the block stays until what may still be
    // under way to it has landed (drain).
    uint32_t limit = a.spin_limit;
    __device__ __forceinline__ bool well() const { return limit != 0; }
    __device__ __forceinline__ void got(bool ok) {
        if (ok) return;
        limit = 0;
        atomicCAS(a.dev_err, kDevOk, (uint32_t)kDevTimeoutCopy);
    }
};

template <typename TIO, int V, int LC, int NW, int ST, int MINB, How HOW>
__global__ void __launch_bounds__(32 * NW, MINB) scan_fwd(ScanArgs a, const __grid_constant__ CUtensorMap mg,
                                                    const __grid_constant__ CUtensorMap mx) {
    using B = Block<V, LC, NW, HOW>;
    using T = typename B::T;
    using P = typename B::P;
    using Sp = Span<V>;
    extern __shared__ __align__(1024) unsigned char slots[];
    __shared__ P wsum[2][NW][32];  // the warps' (s, H)
    __shared__ P csum[2][kMaxCluster][32];
    __shared__ uint64_t bars[(ST ? ST : 1) + 2];
    B k(a);
    Ring<TIO, V, LC * NW, 32 * NW, 2, ST ? ST : 1, HOW> ring{slots, bars + 2, k.c - k.cl, k.b, a.T, a.C,
                                                             a.B * a.T * a.C * (int64_t)sizeof(TIO)};
    Exchange<P> ex{csum, bars};
    const CUtensorMap* const maps[2] = {&mg, &mx};
    const void* const from[2] = {a.g, a.x};
    const int64_t tiles = k.tiles;
    const uint32_t S = k.S, rank = k.rank;
    if (threadIdx.x == 0) {
        ex.init();
        if (ST) ring.init();
        fence_mbar_init();
    }
    if (HOW == kCopy)
        __syncthreads();
    else
        __syncwarp();
    if (S > 1) cluster_arrive();
    grid_dep_wait();  // before any global memory access
    if (ST && ring.mine())
        for (int it = 0; it < ST && (int64_t)it * S + rank < tiles; ++it)
            if (it || (int)rank != a.drop_tile) ring.fetch(it, (it * (int64_t)S + rank) * k.tile, maps, from);
    T carry = k.load_state(a.state_in, k.b);
    if (S > 1) {
        cluster_wait();  // every block of the cluster runs and its barriers are ready
        sync_with(carry);
    } else {
        __syncthreads();
    }

    int it = 0;
    auto stride = [&](auto all, int64_t j, int64_t t0, int n) {
        constexpr bool ALL = decltype(all)::value;
        const int64_t at = (k.b * a.T + t0) * a.C + k.c;
        T sg[LC], x[LC];
        if (ST) {  // a row past T, a channel past C: zeros, or another row's values
            const uint32_t e = (uint32_t)(at - k.cl);
#pragma unroll
            for (int s = 0; s < LC; ++s) {
                sg[s] = ring.get(it, 0, k.wt * LC + s, e + s * (uint32_t)a.C);
                x[s] = ring.get(it, 1, k.wt * LC + s, e + s * (uint32_t)a.C);
            }
        } else {
            const int rows = k.live ? n : 0;
            load_rows<TIO, V, LC, ALL>(static_cast<const TIO*>(a.g) + at, a.C, rows, 0.f, sg);
            load_rows<TIO, V, LC, ALL>(static_cast<const TIO*>(a.x) + at, a.C, rows, 0.f, x);
        }
        T A = Lanes<V>::all(1.f), Dn = Lanes<V>::all(kNoDecay), H = Lanes<V>::all(0.f);
#pragma unroll
        for (int s = 0; s < LC; ++s) {
            sg[s] = gate(sg[s]);
            if (!ALL && s >= n) {  // no such token: the state stays
                sg[s] = Lanes<V>::all(-0.f);
                x[s] = Lanes<V>::all(0.f);
            }
            // the two sums up to each token replace its gate and input: h_t = A_t h_in + H_t
            if (B::kStaged) Dn = vfma(sg[s], A, Dn);
            A = gate_decay(sg[s], A);
            H = gate_step(sg[s], H, x[s]);
            sg[s] = A;
            x[s] = H;
        }
        P(*ws)[32] = wsum[it & 1];
        ws[k.warp][k.lane] = Sp::pack(B::seal(A, Dn), H);
        if (S > 1 && threadIdx.x == 0 && k.well()) ex.expect(it, S);
        __syncthreads();
        if (ST && ring.mine() && k.well() && j + (int64_t)ST * S < tiles)
            ring.fetch(it + ST, (j + (int64_t)ST * S) * k.tile, maps, from);
        // this warp's channels: warps w0 .. w0 + WT - 1 in time order
        const int w0 = ST ? 0 : k.warp - k.wt, WT = ST ? NW : k.WT;
        T h = carry;
        if (B::kStaged && S > 1) {
            // the block's steps before this warp's; the last warp goes on to the block's own sums
            T tA = Lanes<V>::all(1.f), tD = Lanes<V>::all(kNoDecay), tH = Lanes<V>::all(0.f);
            auto fold = [&](int w) {
                const P p = ws[w][k.lane];
                tD = vfma(Sp::gate(p), tA, tD);
                tA = span_decay(Sp::gate(p), tA);
                tH = span_step(Sp::gate(p), Sp::H(p), tH);
            };
#pragma unroll
            for (int w = 0; w < NW - 1; ++w)
                if (w < k.wt) fold(w);
            const T ps = span_gate(tA, tD), pH = tH;
            if (k.wt == NW - 1) {
                fold(NW - 1);
                if (k.well() && (int)rank != a.drop_sums) ex.send(it, S, rank, k.lane, Sp::pack(span_gate(tA, tD), tH));
            }
            k.got(ex.wait(it, k.limit));
            for (uint32_t r = 0; r < S; ++r) {
                if (r == rank) h = carry;
                const P p = csum[it & 1][r][k.lane];
                carry = span_step(Sp::gate(p), Sp::H(p), carry);
            }
            h = span_step(ps, pH, h);
        } else {
#pragma unroll
            for (int w = 0; w < WT; ++w) {
                if (w == k.wt) h = carry;
                const P p = ws[w0 + w][k.lane];
                carry = B::pass(Sp::gate(p), Sp::H(p), carry);
            }
        }
        if (a.carry && t0 < a.T && t0 % kGatedCarrySteps == 0)
            k.store_state(a.carry, k.b * saved_states(a.T) + t0 / kGatedCarrySteps, h);
        TIO* y = static_cast<TIO*>(a.y) + at;
#pragma unroll
        for (int s = 0; s < LC; ++s) {
            if (ALL || s < n) k.store(y + s * a.C, vfma(sg[s], h, x[s]), ALL);
        }
    };
    for (int64_t j0 = 0; j0 < tiles; j0 += S, ++it) {
        // not sooner: the next kernel's waiting blocks would crowd this one's onto fewer SMs when that
        // kernel is this one again (bf16 backward, 4x1024x4096: 37 against 45 us)
        if (j0 + S >= tiles) grid_dep_launch_dependents();
        const int64_t j = j0 + rank, t0 = j * k.tile + k.wt * LC;
        if (ST && j < tiles) k.got(ring.wait(it, k.limit));
        if (k.whole && (j + 1) * k.tile <= a.T)  // the same for every warp of the block
            stride(std::true_type{}, j, t0, LC);
        else
            stride(std::false_type{}, j, t0, t0 < a.T ? (int)min64(LC, a.T - t0) : 0);
    }
    if (ST && !k.well() && ring.mine()) ring.drain(a.spin_limit);
    if (rank == 0 && k.wt == 0) k.store_state(a.state_out, k.b, carry);
    if (S > 1) {  // no block leaves while another may still send to it
        __syncwarp();
        cluster_arrive_relaxed();
        cluster_wait();
        if (!k.well()) ex.drain(a.spin_limit);
    }
}

// Gradients, in reverse time.  With m_t the gradient reaching h_t from the later tokens
// (m_{T-1} = gstate) and lam_t = gy_t + m_t:
//   gx_t = i_t lam_t,  gg_t = f_t i_t (h_{t-1} - x_t) lam_t,  m_{t-1} = f_t lam_t
// A span maps m by m_out = A m_in + M with the forward's A, so the split over warps, blocks and
// strides is the forward's mirrored.  h_{t-1} comes from the tile's saved entering state and the
// forward recurrence of the tile's own steps (the warps' H, exchanged together with M): g, x and
// gy are read once and no other per-token value is needed.  m, lam and M are kept negated: every
// product then is one of s with no sign change on a packed operand.
template <typename TIO, int V, int LC, int NW, int ST, int MINB, How HOW>
__global__ void __launch_bounds__(32 * NW, MINB) scan_bwd(ScanArgs a, const __grid_constant__ CUtensorMap mg,
                                                    const __grid_constant__ CUtensorMap mx,
                                                    const __grid_constant__ CUtensorMap mgy) {
    using B = Block<V, LC, NW, HOW>;
    using T = typename B::T;
    using P = typename B::P;
    using Sp = Span<V>;
    extern __shared__ __align__(1024) unsigned char slots[];
    // gy stays in its slot, in a ring of its own with a slot more than the other's
    constexpr bool kLate = stages_gy_apart<TIO, HOW>;
    constexpr int kST = ST ? ST : 1, kEarly = kLate ? 2 : 3;
    __shared__ P wsum[2][NW][32];  // the warps' (s, H)
    __shared__ T wadj[2][NW][32];  // and M
    __shared__ P csum[2][kMaxCluster][32];
    __shared__ uint64_t bars[2 + kST + (kLate ? kST + 1 : 0)];
    B k(a);
    const int64_t bytes = a.B * a.T * a.C * (int64_t)sizeof(TIO);
    Ring<TIO, V, LC * NW, 32 * NW, kEarly, kST, HOW> ring{slots, bars + 2, k.c - k.cl, k.b, a.T, a.C, bytes};
    Ring<TIO, V, LC * NW, 32 * NW, 1, kST + 1, HOW> late{slots + ST * kEarly * Tile<TIO, V, LC * NW, HOW>::kBytes,
                                                         bars + 2 + kST, k.c - k.cl, k.b, a.T, a.C, bytes};
    Exchange<P> ex{csum, bars};
    const CUtensorMap* const maps[3] = {&mg, &mx, &mgy};
    const void* const from[3] = {a.g, a.x, a.gy};
    const int64_t tiles = k.tiles;
    const uint32_t S = k.S, rank = k.rank;
    if (threadIdx.x == 0) {
        ex.init();
        if (ST) ring.init();
        if (kLate) late.init();
        fence_mbar_init();
    }
    if (HOW == kCopy)
        __syncthreads();
    else
        __syncwarp();
    if (S > 1) cluster_arrive();
    grid_dep_wait();  // before any global memory access
    auto fetch = [&](int it, int64_t j) {
        if (j < 0) return;
        ring.fetch(it, j * k.tile, maps, from);
        if (kLate) late.fetch(it, j * k.tile, maps + 2, from + 2);
    };
    if (ST && ring.mine())
        for (int it = 0; it < ST; ++it)
            if (it || (int)rank != a.drop_tile) fetch(it, tiles - 1 - it * (int64_t)S - rank);
    T carry = neg(k.load_state(a.gstate, k.b));
    const int64_t states0 = k.b * saved_states(a.T);
    if (S > 1) {
        cluster_wait();
        sync_with(carry);
    } else {
        __syncthreads();
    }

    int it = 0;
    auto stride = [&](auto all, int64_t j, int64_t t0, int n) {
        constexpr bool ALL = decltype(all)::value;
        // the block's tile, and this lane's place in it: a 32-bit offset serves every array
        const int64_t tile0 = (k.b * a.T + j * k.tile) * a.C + (k.c - k.cl);
        const uint32_t row = (uint32_t)a.C, off = (uint32_t)(k.wt * LC) * row + (uint32_t)k.cl;
        const uint32_t e = (uint32_t)tile0 + (uint32_t)(k.wt * LC) * row;  // the warp's first row begins here
        T sg[LC], x[LC], gy[LC], As[LC];
        // a tile is a multiple of kGatedCarrySteps long, or holds the whole sequence (j = 0)
        T h = j >= 0 ? k.load_state(a.carry, states0 + j * (LC * NW / kGatedCarrySteps)) : Lanes<V>::all(0.f);
        if (ST) {
#pragma unroll
            for (int s = 0; s < LC; ++s) {
                sg[s] = ring.get(it, 0, k.wt * LC + s, e + s * row);
                x[s] = ring.get(it, 1, k.wt * LC + s, e + s * row);
                if (!kLate) gy[s] = ring.get(it, kEarly - 1, k.wt * LC + s, e + s * row);
            }
        } else {
            const int rows = k.live ? n : 0;
            load_rows<TIO, V, LC, ALL>(static_cast<const TIO*>(a.g) + tile0 + off, a.C, rows, 0.f, sg);
            load_rows<TIO, V, LC, ALL>(static_cast<const TIO*>(a.x) + tile0 + off, a.C, rows, 0.f, x);
            load_rows<TIO, V, LC, ALL>(static_cast<const TIO*>(a.gy) + tile0 + off, a.C, rows, 0.f, gy);
        }
        auto gy_at = [&](int s) {
            if constexpr (kLate) {
                return !ALL && s >= n ? Lanes<V>::all(0.f) : late.get(it, 0, k.wt * LC + s, e + s * row);
            } else {
                return gy[s];
            }
        };
        T A = Lanes<V>::all(1.f), Dn = Lanes<V>::all(kNoDecay), H = Lanes<V>::all(0.f), M = Lanes<V>::all(0.f);
#pragma unroll
        for (int s = 0; s < LC; ++s) {
            sg[s] = gate(sg[s]);
            if (!ALL && s >= n) {
                sg[s] = Lanes<V>::all(-0.f);
                x[s] = Lanes<V>::all(0.f);
                if (!kLate) gy[s] = Lanes<V>::all(0.f);
            }
            // x becomes h_{t-1} - x_t of the span from zero; the state entering adds As_t h_in to it
            As[s] = A;
            A = gate_decay(sg[s], A);
            const T d = vsub(H, x[s]);
            H = vfma(sg[s], d, pick(sg[s], H, x[s]));
            x[s] = d;
        }
        if (kLate && j >= 0) k.got(late.wait(it, k.limit));
#pragma unroll
        for (int s = LC - 1; s >= 0; --s) {
            M = gate_decay(sg[s], vsub(M, gy_at(s)));
            if (B::kStaged) Dn = vfma(sg[s], As[s], Dn);
        }
        P(*ws)[32] = wsum[it & 1];
        T(*wm)[32] = wadj[it & 1];
        ws[k.warp][k.lane] = Sp::pack(B::seal(A, Dn), H);
        wm[k.warp][k.lane] = M;
        if (S > 1 && threadIdx.x == 0 && k.well()) ex.expect(it, S);
        __syncthreads();
        if (ST && ring.mine() && k.well()) fetch(it + ST, j - (int64_t)ST * S);  // gy's slot is the stride's before
        const int w0 = ST ? 0 : k.warp - k.wt, WT = ST ? NW : k.WT;
#pragma unroll
        for (int w = 0; w < WT - 1; ++w)
            if (w < k.wt) {
                const P p = ws[w0 + w][k.lane];
                h = B::pass(Sp::gate(p), Sp::H(p), h);
            }
        T m = carry;
        if (B::kStaged && S > 1) {
            T tA = Lanes<V>::all(1.f), tD = Lanes<V>::all(kNoDecay), tM = Lanes<V>::all(0.f), ps = tD, pM = tM;
#pragma unroll
            for (int w = NW - 1; w >= 0; --w) {
                if (w == k.wt) {  // the block's steps after this warp's
                    ps = span_gate(tA, tD);
                    pM = tM;
                }
                const T sw = Sp::gate(ws[w][k.lane]);
                tD = vfma(sw, tA, tD);
                tA = span_decay(sw, tA);
                tM = span_step(sw, wm[w][k.lane], tM);
            }
            if (k.wt == 0 && k.well() && (int)rank != a.drop_sums) ex.send(it, S, rank, k.lane, Sp::pack(span_gate(tA, tD), tM));
            k.got(ex.wait(it, k.limit));
            for (uint32_t r = 0; r < S; ++r) {
                if (r == rank) m = carry;
                const P p = csum[it & 1][r][k.lane];
                carry = span_step(Sp::gate(p), Sp::H(p), carry);
            }
            m = span_step(ps, pM, m);
        } else {
#pragma unroll
            for (int w = WT - 1; w >= 0; --w) {
                if (w == k.wt) m = carry;
                carry = B::pass(Sp::gate(ws[w0 + w][k.lane]), wm[w0 + w][k.lane], carry);
            }
        }
        TIO *gx = static_cast<TIO*>(a.y) + tile0, *gg = static_cast<TIO*>(a.gg) + tile0;
#pragma unroll
        for (int s = LC - 1; s >= 0; --s) {
            const T lam = vsub(m, gy_at(s));  // negated, as m
            T in;
            m = gate_split(sg[s], lam, in);
            const T out = vmul(vmul(gate_slope_neg(sg[s]), vfma(As[s], h, x[s])), lam);
            if (ALL || s < n) {
                k.store(gx + off + s * row, in, ALL);
                k.store(gg + off + s * row, out, ALL);
            }
        }
    };
    for (int64_t j0 = 0; j0 < tiles; j0 += S, ++it) {
        if (j0 + S >= tiles) grid_dep_launch_dependents();  // not sooner, as in the forward
        const int64_t j = tiles - 1 - j0 - rank;  // < 0: past the sequence's start
        const int64_t t0 = j * k.tile + k.wt * LC;
        if (ST && j >= 0) k.got(ring.wait(it, k.limit));
        if (k.whole && j >= 0 && (j + 1) * k.tile <= a.T)
            stride(std::true_type{}, j, t0, LC);
        else
            stride(std::false_type{}, j, t0, j >= 0 && t0 < a.T ? (int)min64(LC, a.T - t0) : 0);
    }
    if (ST && !k.well() && ring.mine()) {
        ring.drain(a.spin_limit);
        if (kLate) late.drain(a.spin_limit);
    }
    if (rank == 0 && k.wt == 0) k.store_state(a.state_out, k.b, neg(carry));
    if (S > 1) {
        __syncwarp();
        cluster_arrive_relaxed();
        cluster_wait();
        if (!k.well()) ex.drain(a.spin_limit);
    }
}

// Many channels: a warp walks the whole sequence of 32 V channels, U rows at a time, with nothing to
// exchange.  `groups` counts groups of 32 V channels.
template <int V>
struct Rows {
    using T = typename Lanes<V>::T;
    const ScanArgs& a;
    int64_t b, c;
    bool live;

    __device__ __forceinline__ Rows(const ScanArgs& args) : a(args) {
        const int64_t unit = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
        b = unit / a.groups;
        c = (unit % a.groups) * (32 * V) + (threadIdx.x & 31) * V;
        live = b < a.B && c < a.C;
    }
    __device__ __forceinline__ T load(const float* p, int64_t row) const {
        float t[V];
#pragma unroll
        for (int q = 0; q < V; ++q) t[q] = 0.f;
        if (p) Vec<float, V>::load(p + row * a.C + c, t);
        return Lanes<V>::make(t);
    }
    template <typename TO>
    __device__ __forceinline__ void store(TO* p, T v) const {
        float t[V];
        Lanes<V>::split(v, t);
        Vec<TO, V>::store(p, t);
    }
};

template <typename TIO, int V, int U>
__global__ void __launch_bounds__(128) rows_fwd(ScanArgs a) {
    using T = typename Lanes<V>::T;
    const Rows<V> k(a);
    grid_dep_wait();  // before any global memory access
    if (k.live) {
        const int64_t at = k.b * a.T * a.C + k.c;
        T h = k.load(a.state_in, k.b);
        auto rows = [&](auto all, int64_t t0, int n) {
            constexpr bool ALL = decltype(all)::value;
            T s[U], x[U];
            load_rows<TIO, V, U, ALL>(static_cast<const TIO*>(a.g) + at + t0 * a.C, a.C, n, 0.f, s);
            load_rows<TIO, V, U, ALL>(static_cast<const TIO*>(a.x) + at + t0 * a.C, a.C, n, 0.f, x);
            if (a.carry && t0 % kGatedCarrySteps == 0)
                k.store(a.carry + (k.b * saved_states(a.T) + t0 / kGatedCarrySteps) * a.C + k.c, h);
            TIO* y = static_cast<TIO*>(a.y) + at + t0 * a.C;
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (ALL || i < n) {
                    h = gate_step(gate(s[i]), h, x[i]);
                    k.store(y + i * a.C, h);
                }
        };
        int64_t t0 = 0;
        for (; t0 + U <= a.T; t0 += U) rows(std::true_type{}, t0, U);
        if (t0 < a.T) rows(std::false_type{}, t0, (int)(a.T - t0));
        if (a.state_out) k.store(a.state_out + k.b * a.C + k.c, h);
    }
    grid_dep_launch_dependents();
}

// At most kGatedCarrySteps steps, walked forward for s and h_{t-1} - x_t, which wait in shared memory (a
// lane reads only what it wrote), and then backward.
template <typename TIO, int V, int U>
__global__ void __launch_bounds__(128) rows_bwd(ScanArgs a) {
    using T = typename Lanes<V>::T;
    using P = typename Span<V>::P;
    using Sp = Span<V>;
    extern __shared__ __align__(1024) unsigned char slots[];
    const Rows<V> k(a);
    grid_dep_wait();  // before any global memory access
    if (k.live) {
        const int steps = (int)a.T;
        P* const kept = reinterpret_cast<P*>(slots) + (threadIdx.x >> 5) * steps * 32 + (threadIdx.x & 31);
        const int64_t at = k.b * a.T * a.C + k.c;
        T m = neg(k.load(a.gstate, k.b)), h = k.load(a.carry, k.b);
        auto forward = [&](auto all, int t0, int n) {
            constexpr bool ALL = decltype(all)::value;
            T s[U], x[U];
            load_rows<TIO, V, U, ALL>(static_cast<const TIO*>(a.g) + at + (int64_t)t0 * a.C, a.C, n, 0.f, s);
            load_rows<TIO, V, U, ALL>(static_cast<const TIO*>(a.x) + at + (int64_t)t0 * a.C, a.C, n, 0.f, x);
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (ALL || i < n) {
                    const T sg = gate(s[i]), d = vsub(h, x[i]);
                    kept[(t0 + i) * 32] = Sp::pack(sg, d);
                    h = vfma(sg, d, pick(sg, h, x[i]));
                }
        };
        auto backward = [&](auto all, int t0, int n) {
            constexpr bool ALL = decltype(all)::value;
            T gy[U];
            load_rows<TIO, V, U, ALL>(static_cast<const TIO*>(a.gy) + at + (int64_t)t0 * a.C, a.C, n, 0.f, gy);
            TIO *gx = static_cast<TIO*>(a.y) + at + (int64_t)t0 * a.C, *gg = static_cast<TIO*>(a.gg) + at + (int64_t)t0 * a.C;
#pragma unroll
            for (int i = U - 1; i >= 0; --i)
                if (ALL || i < n) {
                    const P p = kept[(t0 + i) * 32];
                    const T sg = Sp::gate(p), lam = vsub(m, gy[i]);  // negated, as m
                    T in;
                    m = gate_split(sg, lam, in);
                    k.store(gx + i * a.C, in);
                    k.store(gg + i * a.C, vmul(vmul(gate_slope_neg(sg), Sp::H(p)), lam));
                }
        };
        const int whole = steps / U * U;
        for (int t0 = 0; t0 < whole; t0 += U) forward(std::true_type{}, t0, U);
        if (whole < steps) {
            forward(std::false_type{}, whole, steps - whole);
            backward(std::false_type{}, whole, steps - whole);
        }
        for (int t0 = whole - U; t0 >= 0; t0 -= U) backward(std::true_type{}, t0, U);
        if (a.state_out) k.store(a.state_out + k.b * a.C + k.c, neg(m));
    }
    grid_dep_launch_dependents();
}

// One token per row-channel: h <- f h + i x, y = h, one 16-byte vector of g per thread.  Bound by the
// bytes of g, x, y and the state in and out: 256x32x4096 fp32 98 us, 6870 GB/s (a grid of eight
// blocks per SM walking the rows took 114).
template <typename TIO, int V>
__global__ void __launch_bounds__(256) step_kernel(int64_t n, const TIO* __restrict__ g, const TIO* __restrict__ x,
                                                   float* __restrict__ state, TIO* __restrict__ y) {
    constexpr int VS = V < 4 ? V : 4;  // channels per access of the state
    grid_dep_launch_dependents();
    grid_dep_wait();  // before any global memory access
    const int64_t stride = (int64_t)gridDim.x * blockDim.x * V;
    for (int64_t k = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * V; k < n; k += stride) {
        float gv[V], xv[V], h[V / VS][VS];
        Vec<TIO, V>::load(g + k, gv);
        Vec<TIO, V>::load(x + k, xv);
#pragma unroll
        for (int q = 0; q < V / VS; ++q) Vec<float, VS>::load(state + k + q * VS, h[q]);
#pragma unroll
        for (int q = 0; q < V; ++q) {
            float& hq = h[q / VS][q % VS];
            hq = gate_step(gate(gv[q]), hq, xv[q]);
            gv[q] = hq;
        }
#pragma unroll
        for (int q = 0; q < V / VS; ++q) Vec<float, VS>::store(state + k + q * VS, h[q]);
        Vec<TIO, V>::store(y + k, gv);
    }
}

__global__ void copy_or_zero(int64_t n, const float* in, float* out) {
    grid_dep_launch_dependents();
    grid_dep_wait();  // before any global memory access
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
        out[i] = in ? in[i] : 0.f;
}

int sm_count() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

// Clusters of S blocks of a kernel that are resident at once (asked once per kernel and device): they
// lie within a GPC, so S blocks of every eight GPCs' 18 or 20 SMs do not always come out even.
struct ClusterRoom {
    std::atomic<int> of[64][kMaxCluster + 1] = {};

    template <typename K>
    int operator()(int dev, K kern, cudaLaunchConfig_t cfg, int S) {
        if (dev < 0 || dev >= 64) return 0;
        int known = of[dev][S].load(std::memory_order_relaxed);  // the answer + 1
        if (known == 0) {
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim = {(unsigned)S, 1, 1};
            cfg.gridDim = dim3((unsigned)S);
            cfg.attrs = at;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes) != cudaSuccess ||
                cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
                cudaGetLastError();  // no cluster of this size
                n = 0;
            }
            of[dev][S].store(known = n + 1, std::memory_order_relaxed);
        }
        return known - 1;
    }
};

// One configuration: V channels per lane, LC steps per warp, NW warps per block, ST staged tiles,
// RES blocks resident per SM; its launch for one shape.
template <typename TIO, int V, int LC, int NW, int ST, int RES, bool BWD, How HOW = kTma>
struct ScanLaunch {
    static constexpr int kArrays = BWD ? 3 : 2;
    static constexpr int kTiles = (ST * kArrays + (BWD && stages_gy_apart<TIO, HOW>)) * Tile<TIO, V, LC * NW, HOW>::kBytes;
    // one block per SM where the rules below count on it, however few registers it takes
    static constexpr int kSmem = RES == 1 && kTiles < 116 * 1024 ? 116 * 1024 : kTiles;
    static_assert((ST > 0) == (HOW != kDirect), "direct loads stage nothing");

    int wt_log = 0, S = 0;  // log2 of the warps along time, blocks per cluster
    int64_t groups = 0, units = 0, strides = 0;
    bool capped = false;  // a cluster could not have more blocks, where there was room for them
    cudaLaunchConfig_t cfg = {};

    static constexpr auto kernel() {
        if constexpr (BWD)
            return scan_bwd<TIO, V, LC, NW, ST, RES, HOW>;
        else
            return scan_fwd<TIO, V, LC, NW, ST, RES, HOW>;
    }

    explicit ScanLaunch(const GatedScanShape& s) {
        while ((1 << wt_log) < NW && (ST || (int64_t)(LC << wt_log) < s.T)) ++wt_log;
        const int64_t W = (int64_t)(NW >> wt_log) * 32 * V, tiles = (s.T + LC * NW - 1) / (LC * NW);
        groups = (s.C + W - 1) / W;
        units = s.B * groups;
        cfg.blockDim = dim3(32 * NW);
        cfg.dynamicSmemBytes = kSmem;
        int dev = -1;
        cudaGetDevice(&dev);
        // the most blocks per cluster with every cluster resident at once, then the fewest that walk
        // the sequence in as many strides
        static ClusterRoom room;
        S = (int)min64(kMaxCluster, tiles);
        while (S > 1 && units > room(dev, kernel(), cfg, S)) --S;
        capped = S == kMaxCluster && tiles > kMaxCluster;
        strides = (tiles + S - 1) / S;
        S = (int)((tiles + strides - 1) / strides);
    }

    cudaError_t operator()(const GatedScanShape& s, ScanArgs a, cudaStream_t stream) {
        if (kSmem > 0)
            if (cudaError_t e = cudaFuncSetAttribute(kernel(), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) return e;
        a.wt_log = wt_log;
        a.groups = groups;
        CUtensorMap m[3] = {};
        if (HOW == kTma) {
            const void* from[3] = {a.g, a.x, a.gy};
            for (int k = 0; k < kArrays; ++k)
                if (!make_tile_map(&m[k], from[k], s.B, s.T, s.C, s.io, 32 * V, LC * NW)) return cudaErrorInvalidValue;
        }
        cfg.stream = stream;
        cfg.gridDim = dim3((unsigned)(units * S));
        cudaLaunchAttribute at[2];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = kProgrammaticLaunch ? 1 : 0;
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim = {(unsigned)S, 1, 1};
        cfg.attrs = at;
        cfg.numAttrs = S > 1 ? 2 : 1;
        if constexpr (BWD)
            return cudaLaunchKernelEx(&cfg, kernel(), a, m[0], m[1], m[2]);
        else
            return cudaLaunchKernelEx(&cfg, kernel(), a, m[0], m[1]);
    }
};

template <typename TIO, int V, int LC, int NW, int ST, int RES, bool BWD, How HOW = kTma>
cudaError_t launch_scan(const GatedScanShape& s, const ScanArgs& a, cudaStream_t stream) {
    return ScanLaunch<TIO, V, LC, NW, ST, RES, BWD, HOW>(s)(s, a, stream);
}

// Bytes of the steps that a warp of rows_bwd keeps in shared memory, at the most: two such warps, or four of
// half, take 32 KB, which a block has without asking.
constexpr int kRowsKept = 16384;

// One warp per sequence and 32 V channels (backward: T <= kGatedCarrySteps).
template <typename TIO, int V, int U, bool BWD>
cudaError_t launch_rows(const GatedScanShape& s, ScanArgs a, cudaStream_t stream) {
    a.groups = (s.C + 32 * V - 1) / (32 * V);
    const int kept = BWD ? (int)s.T * 32 * (int)sizeof(typename Span<V>::P) : 0;  // bytes per warp
    const int warps = kept > kRowsKept / 2 ? 2 : 4;
    const dim3 grid((unsigned)((s.B * a.groups + warps - 1) / warps));
    if constexpr (BWD)
        return launch_pdl(rows_bwd<TIO, V, U>, grid, dim3(32 * warps), warps * kept, stream, a);
    else
        return launch_pdl(rows_fwd<TIO, V, U>, grid, dim3(32 * warps), 0, stream, a);
}

// Times below: us on a B200 in a CUDA graph, inputs over the L2, shapes B x T x C.  Those of staged forms were
// taken before spans carried 1 - A (span_gate): both sides of a comparison are up to 4% (forward) and 7%
// (backward) slower since.
//
// Sequences of at most kShort steps are read directly: 64x32x2048 fp32 takes 33 staged and 13 direct
// (a short tile leaves warps idle), 32x128x2048 20 and 21, 8x1024x768 15 and 26.  The bf16 backward's
// staged tile is 64 steps: from 33 on it wins (32x48x768 7.1 against 10.5, 64x64x768 11 against 15).
constexpr int64_t kShort = 64, kShortHalfBackward = 32;

// Short sequences of many channels: one warp per sequence and 32 or 64 channels instead (rows_fwd,
// rows_bwd), at 16 warps of pairs per SM for T < 256 forward: 256x32x4096 fp32 64 against 83 direct
// (bf16 35 against 75), 256x65x4096 129 against 286 staged (71 against 243), 40x200x4096 62 against 74
// (42 against 63), but 40x1024x4096 326 against 315 (204 against 155).  With fewer warps single
// channels, T < 128: 64x48x768 7.3 against 12.1, 32x128x1280 14.7 against 14.2, 16x48x1024 5.2 against
// 4.8.  Backward, with the steps kept in shared memory: pairs for the shortest (256x8x4096 28 against
// 34, bf16 19 against 33; 256x24x4096 58 in bf16, 92 by single channels), then single channels
// (256x24x4096 93, 256x48x4096 197 against 279, bf16 139 against 268, or 169 staged); fp32 not at 32 and 64
// steps, where the direct form is the faster (256x32x4096 123 against 132, 256x64x4096 255 against 274;
// at 16 it is not, 65 against 56), bf16 not where tiles of 64 steps are staged nearly full (256x56x4096
// 173 against 222).
constexpr int64_t kRowsForward = 256, kRowsForwardFew = 128, kRowsBackward = kGatedCarrySteps;

// Rows that TMA can stage: 4x1024x2048 forward 19, backward 33, in bf16 13 and 26.  Others are staged
// by copies: 4x1024x2049 25, 42, 20 and 31 (direct loads took 25, 91, 46 and 71).
bool tma_rows(const GatedScanShape& s) {
    const int64_t es = s.io == 1 ? 2 : 4;
    return s.C * es % 16 == 0 && s.T <= INT32_MAX &&
           s.T * s.C * es < (int64_t(1) << 40);  // a tensor map's coordinates and strides
}

// fp32: pairs per lane halve the instructions, single channels make twice the blocks.  Pairs win on
// long sequences where their blocks, in clusters of at most four, fill three quarters of the SMs, one
// each and all at once (1x16384x4096: forward 118 against 151, backward 210 against 264;
// 1x16384x2048: 61 against 76, 111 against 125; 1x16384x1792: 61 against 66, 107 against 114), single
// channels elsewhere (8x1024x768: 15.0 against 16.3, 25.1 against 27.3; 4x4096x768: 28 against 32, 52
// against 57; 1x16384x5120: 187 against 198, 312 against 347; in clusters of five, 2x4096x768: 15
// against 18, 27 against 29).  Just on either side of the rule the two are within a tenth of each other.
//
// Few channels: a cluster ends at eight blocks and the SMs are not filled, so what counts is how many
// strides the sequence takes.  A tile of 256 steps takes the fewest while there is an SM for each of
// its blocks: forward fp32 (bf16), 1x16384x64 16 against 21 (15 against 28), x768 28 against 32 (25
// against 34), x1024 33 against 35 (29 against 38); backward 28 against 32 (28 against 59), 50
// against 52 (46 against 70).  The bf16 backward, whose tile otherwise is 64 steps, has one of 128 in
// between: pairs, or single channels where those take fewer strides (1x16384x1536 pairs 75, single
// channels 85, the tile of 64 80; 1x4096x768 14.6, 15.2, 19; 2x1000x512 9.2, 6.6, 8.2).  Rows staged by
// copies likewise: forward 1x16384x257 32 against 39 (30 against 47), x769 51 against 56 (48, 48);
// backward tile 128 50 against 71, 83 against 91, 256 (43 against 94, 69 against 95).
constexpr int64_t kLong = 4096;

template <typename LAUNCH>
bool one_per_sm(const LAUNCH& l) {
    return l.units * l.S <= sm_count();
}
template <typename LAUNCH>
bool fills_once(const LAUNCH& l) {
    return one_per_sm(l) && l.S <= 4 && l.units * l.S * 4 >= (int64_t)sm_count() * 3;
}

// Direct: a block's warps hold the whole sequence, a warp no more steps than it needs (512x1x4096
// fp32 with 8 steps per warp: 38).
template <typename TIO, int V, bool BWD>
cudaError_t launch_direct(const GatedScanShape& s, const ScanArgs& a, cudaStream_t stream) {
    if (s.T == 1) return launch_scan<TIO, V, 1, 4, 0, 4, BWD, kDirect>(s, a, stream);
    if (s.T <= 4) return launch_scan<TIO, V, 4, 4, 0, 4, BWD, kDirect>(s, a, stream);
    if (s.T <= 32) return launch_scan<TIO, V, 8, 4, 0, 4, BWD, kDirect>(s, a, stream);
    return launch_scan<TIO, V, 8, 8, 0, 2, BWD, kDirect>(s, a, stream);
}

// The forward's staged form: 32 steps per warp and four warps (fewer summaries to fold: bf16
// 4x4096x2048 38 against 43 with 16 steps and eight warps).  The backward holds four values per
// token, which 32 steps spill: 16 steps, eight warps.  bf16 always in pairs (a row of the tile is
// then 128 bytes: forward 38 against 54); its backward leaves gy in the staged tile, so that more
// blocks fit an SM: three of four warps (64x1024x768 91, 8x1024x768 17.1, 4x1024x4096 37), two of
// four with three tiles staged (103, 22.1, 36.4), two of eight (119, 21.5, 42).
template <typename TIO, bool BWD>
cudaError_t dispatch_scan(const GatedScanShape& s, const ScanArgs& a, cudaStream_t stream) {
    constexpr bool kHalf = sizeof(TIO) == 2;
    const bool tma = tma_rows(s);
    const int64_t singles = s.B * ((s.C + 31) / 32), sms = sm_count();
    const int64_t pairs = s.C % 2 == 0 ? s.B * ((s.C + 63) / 64) : 0;
    if constexpr (BWD) {
        constexpr int64_t kPairs = kHalf ? 32 : 15;
        static_assert(kPairs * 32 * sizeof(Span<2>::P) <= kRowsKept && kRowsBackward * 32 * sizeof(Span<1>::P) <= kRowsKept,
                      "launch_rows has two warps to a block at the least");
        if (pairs >= 16 * sms && s.T <= kPairs) return launch_rows<TIO, 2, 8, true>(s, a, stream);
        if (singles >= 8 * sms && s.T > 8 && s.T <= (kHalf && tma ? 48 : kRowsBackward) && (kHalf || s.T % 32 != 0))
            return launch_rows<TIO, 1, 16, true>(s, a, stream);
    } else {
        if (pairs >= 16 * sms && s.T < kRowsForward) return launch_rows<TIO, 2, 8, false>(s, a, stream);
        if (singles >= 5 * sms && s.T > 8 && s.T < kRowsForwardFew) return launch_rows<TIO, 1, 16, false>(s, a, stream);
    }
    if (s.T <= (BWD && kHalf && tma ? kShortHalfBackward : kShort))
        return s.C % 2 == 0 ? launch_direct<TIO, 2, BWD>(s, a, stream) : launch_direct<TIO, 1, BWD>(s, a, stream);
    if (tma) {
        if constexpr (!kHalf)
            if (s.T >= kLong) {
                ScanLaunch<TIO, 2, BWD ? 16 : 32, BWD ? 8 : 4, 2, 1, BWD> pairs(s);
                if (fills_once(pairs)) return pairs(s, a, stream);
            }
        if constexpr (!BWD) {
            ScanLaunch<TIO, kHalf ? 2 : 1, 32, 4, 2, kHalf ? 2 : 3, false> base(s);
            if (base.strides > 1) {
                ScanLaunch<TIO, 1, 32, 8, 2, 1, false> tall(s);
                if (one_per_sm(tall) && tall.strides <= base.strides) return tall(s, a, stream);
            }
            return base(s, a, stream);
        } else {
            ScanLaunch<TIO, 1, 16, 8, 2, 2, true> mid(s);
            if constexpr (kHalf) {
                ScanLaunch<TIO, 2, 16, 4, 2, 3, true> base(s);
                if (!base.capped) return base(s, a, stream);
            }
            if (mid.strides > 1) {
                ScanLaunch<TIO, 1, 16, 16, 2, 1, true> tall(s);
                if (one_per_sm(tall) && tall.strides < mid.strides) return tall(s, a, stream);
            }
            if constexpr (kHalf) {
                ScanLaunch<TIO, 2, 16, 8, 2, 2, true> pairs(s);
                if (pairs.strides <= mid.strides) return pairs(s, a, stream);
            }
            return mid(s, a, stream);
        }
    }
    // by copies: as above, the backward in tiles of 64 steps, three staged
    if constexpr (!BWD) {
        ScanLaunch<TIO, kHalf ? 2 : 1, 16, 8, 2, 2, false, kCopy> base(s);
        if (base.strides > 1) {
            ScanLaunch<TIO, 1, 16, 16, 2, 1, false, kCopy> tall(s);
            if (one_per_sm(tall) && tall.strides < base.strides) return tall(s, a, stream);
        }
        return base(s, a, stream);
    } else {
        ScanLaunch<TIO, kHalf ? 2 : 1, 16, 4, 3, 2, true, kCopy> base(s);
        if (base.capped) {
            ScanLaunch<TIO, 1, 16, 8, 2, kHalf ? 2 : 1, true, kCopy> mid(s);
            if constexpr (kHalf) {  // in fp32 a tile of 256 steps does not fit
                ScanLaunch<TIO, 1, 16, 16, 2, 1, true, kCopy> tall(s);
                if (one_per_sm(tall) && tall.strides < mid.strides) return tall(s, a, stream);
            }
            if (mid.strides < base.strides) return mid(s, a, stream);
        }
        return base(s, a, stream);
    }
}

// blocks of 256 threads, one unit each (more units than a grid holds: the kernels loop)
unsigned flat_blocks(int64_t units) {
    const int64_t b = (units + 255) / 256;
    return (unsigned)(b < INT32_MAX ? b : INT32_MAX);
}

}  // namespace

bool gated_scan_fits(const GatedScanShape& s) {
    if (s.C > INT32_MAX / 256) return false;  // a tile's offsets are 32-bit
    // the most blocks any split takes: every 32 channels of every sequence, kMaxCluster deep
    return s.B <= INT32_MAX / kMaxCluster / ((s.C + 31) / 32);
}

cudaError_t launch_gated_scan_forward(const GatedScanShape& s, const void* g, const void* x, const float* state_in,
                                      void* y, float* state_out, float* carry, cudaStream_t stream,
                                      const GatedScanWaits& waits) {
    if (s.T == 0)
        return state_out ? launch_pdl(copy_or_zero, dim3(flat_blocks(s.B * s.C)), dim3(256), 0, stream, s.B * s.C,
                                      state_in, state_out)
                         : cudaSuccess;
    ScanArgs a = {};
    a.B = s.B;
    a.T = s.T;
    a.C = s.C;
    a.g = g;
    a.x = x;
    a.state_in = state_in;
    a.y = y;
    a.state_out = state_out;
    a.carry = carry;
    a.dev_err = device_status_word();
    if (!a.dev_err) return cudaGetLastError();
    a.spin_limit = waits.spin_limit;
    a.drop_sums = (int16_t)waits.drop_sums;
    a.drop_tile = (int16_t)waits.drop_tile;
    return s.io == 1 ? dispatch_scan<__nv_bfloat16, false>(s, a, stream) : dispatch_scan<float, false>(s, a, stream);
}

cudaError_t launch_gated_scan_backward(const GatedScanShape& s, const void* g, const void* x, const float* carry,
                                       const void* gy, const float* gstate_out, void* gg, void* gx, float* gstate_in,
                                       cudaStream_t stream, const GatedScanWaits& waits) {
    if (s.T == 0)
        return gstate_in ? launch_pdl(copy_or_zero, dim3(flat_blocks(s.B * s.C)), dim3(256), 0, stream, s.B * s.C,
                                      gstate_out, gstate_in)
                         : cudaSuccess;
    ScanArgs a = {};
    a.B = s.B;
    a.T = s.T;
    a.C = s.C;
    a.g = g;
    a.x = x;
    a.gy = gy;
    a.gstate = gstate_out;
    a.y = gx;
    a.gg = gg;
    a.state_out = gstate_in;
    a.carry = const_cast<float*>(carry);
    a.dev_err = device_status_word();
    if (!a.dev_err) return cudaGetLastError();
    a.spin_limit = waits.spin_limit;
    a.drop_sums = (int16_t)waits.drop_sums;
    a.drop_tile = (int16_t)waits.drop_tile;
    return s.io == 1 ? dispatch_scan<__nv_bfloat16, true>(s, a, stream) : dispatch_scan<float, true>(s, a, stream);
}

cudaError_t launch_gated_scan_step(int64_t n, int io, const void* g, const void* x, float* state, void* y,
                                   cudaStream_t s) {
    if (io == 1) {
        const __nv_bfloat16 *gg = static_cast<const __nv_bfloat16*>(g), *xx = static_cast<const __nv_bfloat16*>(x);
        __nv_bfloat16* yy = static_cast<__nv_bfloat16*>(y);
        if (n % 8 == 0)
            return launch_pdl(step_kernel<__nv_bfloat16, 8>, dim3(flat_blocks(n / 8)), dim3(256), 0, s, n, gg, xx, state, yy);
        return launch_pdl(step_kernel<__nv_bfloat16, 1>, dim3(flat_blocks(n)), dim3(256), 0, s, n, gg, xx, state, yy);
    }
    const float *gg = static_cast<const float*>(g), *xx = static_cast<const float*>(x);
    float* yy = static_cast<float*>(y);
    if (n % 4 == 0)
        return launch_pdl(step_kernel<float, 4>, dim3(flat_blocks(n / 4)), dim3(256), 0, s, n, gg, xx, state, yy);
    return launch_pdl(step_kernel<float, 1>, dim3(flat_blocks(n)), dim3(256), 0, s, n, gg, xx, state, yy);
}

}  // namespace wkvb
