// Gated linear recurrence, per channel (declarations and contract in include/wkv.h):
//   f_t = sigma(g_t), i_t = 1 - f_t = sigma(-g_t),   h_t = f_t h_{t-1} + i_t x_t,   y_t = h_t
//
// A span of steps maps the state entering it to the state leaving it by
//   h_out = A h_in + H,   A = prod f_t,   H = the span's state from zero,
// and two adjacent spans compose as (A1 A2, A2 H1 + H2), so the long axis is split: a warp
// takes kLC consecutive steps of 32 V adjacent channels into registers, sums them up as (A, H),
// and once it knows the state entering its steps runs them again from the registers.  The
// warps of a block cover a tile of kTile steps, the blocks of a cluster adjacent tiles; a
// cluster walks its channels' sequence in strides of S tiles and carries the state from stride
// to stride.  Summaries meet in (distributed) shared memory behind the hardware barriers, in a
// fixed order: no workspace, no waiting on other clusters, and the same bits on every run.
//
// Arithmetic: fp32 whatever the I/O type.  A gate is kept as the smaller of (f, i) with the sign
// of g, from e = 2^(-|g| log2 e) as e / (1 + e), relatively accurate at
// both ends.  A step starts from whichever of h, x it stays near:
//   i <= 1/2:  h + i (x - h)   where a gate holds for thousands of tokens f rounds to within
//                              2^-24 of 1, and repeating f h would drift by that every step;
//   f <  1/2:  x + f (h - x)   a closing gate leaves no rounding of the old state (f = 0: h = x).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "wkv_device.cuh"
#include "wkv_gated_internal.h"
#include "wkv_internal.h"
#include "wkv_vec.cuh"

namespace wkvb {
namespace {

constexpr int kLC = 8;                    // steps per warp
constexpr int kNW = 16;                   // warps per block
constexpr int kThreads = 32 * kNW;
constexpr int kTile = kLC * kNW;          // steps per tile
constexpr int kMaxCluster = 8;            // portable cluster size
static_assert(kTile == kGatedCarrySteps, "one saved state per tile");

struct ScanArgs {
    int64_t B, T, C;
    int64_t groups;  // channel groups per sequence
    int wt_log;      // log2 of the warps of a block along time (kNW unless a shorter tile holds T)
    const void *g, *x, *gy;
    const float* state_in;   // forward: [B][C] or null
    void* y;                 // forward: y; backward: gx
    void* gg;                // backward
    float* state_out;        // forward: state_out; backward: gstate_in; [B][C] or null
    float* carry;            // [B][tiles][C]: forward writes (or null), backward reads
    const float* gstate;     // backward: gradient of state_out, [B][C] or null
};

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
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// this block's shared address as the same place in block `rank` of the cluster
__device__ __forceinline__ void st_cluster_f2(uint32_t saddr, uint32_t rank, float2 v) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(r), "f"(v.x), "f"(v.y) : "memory");
}

// The signed gate: +i where i = sigma(-g) <= 1/2, -f where f = sigma(g) < 1/2 (the sign is g's,
// also on a zero).
__device__ __forceinline__ float signed_gate(float g) {
    const float e = ex2(-fabsf(g) * kLog2e);
    return copysignf(e * rcp(1.f + e), g);
}
__device__ __forceinline__ bool holds(float s) { return __float_as_int(s) >= 0; }  // i <= 1/2

// f h + i x
__device__ __forceinline__ float gate_step(float s, float h, float x) { return fmaf(s, x - h, holds(s) ? h : x); }
// f a
__device__ __forceinline__ float gate_decay(float s, float a) { return fmaf(-s, a, holds(s) ? a : 0.f); }
// i a
__device__ __forceinline__ float gate_input(float s, float a) { return fmaf(s, a, holds(s) ? 0.f : a); }

// V adjacent channels of kLC rows (row stride C elements) as fp32; rows from n on are not read and
// come back as `fill`
template <typename TIO, int V>
__device__ __forceinline__ void load_rows(const TIO* p, int64_t C, int n, float fill, float (&o)[kLC][V]) {
#pragma unroll
    for (int s = 0; s < kLC; ++s) {
#pragma unroll
        for (int q = 0; q < V; ++q) o[s][q] = fill;
        if (s < n) Vec<TIO, V>::load(p + s * C, o[s]);
    }
}

template <typename TIO, int V>
__global__ void __launch_bounds__(kThreads) scan_fwd(ScanArgs a) {
    __shared__ float2 wsum[2][kNW * 32 * V];           // the warps' (A, H), [time warp][channel]
    __shared__ float2 csum[2][kMaxCluster][32 * V];    // the cluster's blocks' (A, H)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int WT = 1 << a.wt_log, wt = warp & (WT - 1), wc = warp >> a.wt_log;
    const int W = (kNW >> a.wt_log) * 32 * V;          // channels of this block
    const int cl = (wc * 32 + lane) * V;               // this lane's first, within the block
    const uint32_t S = cluster_size(), rank = cluster_rank();
    const int64_t unit = blockIdx.x / S, b = unit / a.groups;
    const int64_t c = (unit % a.groups) * W + cl;
    const bool live = c < a.C;
    const int64_t tile = (int64_t)WT * kLC, tiles = (a.T + tile - 1) / tile;
    grid_dep_launch_dependents();
    if (S > 1) cluster_arrive();
    grid_dep_wait();  // before any global memory access
    float carry[V];
#pragma unroll
    for (int q = 0; q < V; ++q) carry[q] = live && a.state_in ? a.state_in[b * a.C + c + q] : 0.f;
    if (S > 1) cluster_wait();  // every block of the cluster runs: its shared memory may be written

    int buf = 0;
    for (int64_t j0 = 0; j0 < tiles; j0 += S, buf ^= 1) {
        const int64_t j = j0 + rank, t0 = j * tile + wt * kLC;
        const int n = live && t0 < a.T ? (int)min64(kLC, a.T - t0) : 0;
        const int64_t at = (b * a.T + t0) * a.C + c;
        float sg[kLC][V], x[kLC][V];
        load_rows<TIO, V>(static_cast<const TIO*>(a.g) + at, a.C, n, INFINITY, sg);  // i = 0: the state stays
        load_rows<TIO, V>(static_cast<const TIO*>(a.x) + at, a.C, n, 0.f, x);
        float A[V], H[V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
            A[q] = 1.f;
            H[q] = 0.f;
        }
#pragma unroll
        for (int s = 0; s < kLC; ++s)
#pragma unroll
            for (int q = 0; q < V; ++q) {
                sg[s][q] = signed_gate(sg[s][q]);
                A[q] = gate_decay(sg[s][q], A[q]);
                H[q] = gate_step(sg[s][q], H[q], x[s][q]);
            }
#pragma unroll
        for (int q = 0; q < V; ++q) wsum[buf][wt * W + cl + q] = make_float2(A[q], H[q]);
        __syncthreads();
        if (S > 1) {
            if (wt == 0) {  // the block's (A, H), to every block of the cluster
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    float2 tot = make_float2(1.f, 0.f);
                    for (int k = 0; k < WT; ++k) {
                        const float2 r = wsum[buf][k * W + cl + q];
                        tot = make_float2(tot.x * r.x, fmaf(r.x, tot.y, r.y));
                    }
                    const uint32_t at_s = smem_u32(&csum[buf][rank][cl + q]);
                    for (uint32_t k = 0; k < S; ++k) st_cluster_f2(at_s, k, tot);
                }
            }
            cluster_arrive();
            cluster_wait();
        }
        float h[V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
            h[q] = carry[q];
            if (S > 1) {
                for (uint32_t k = 0; k < S; ++k) {
                    const float2 r = csum[buf][k][cl + q];
                    carry[q] = fmaf(r.x, carry[q], r.y);
                    if (k + 1 == rank) h[q] = carry[q];
                }
                for (int k = 0; k < wt; ++k) {
                    const float2 r = wsum[buf][k * W + cl + q];
                    h[q] = fmaf(r.x, h[q], r.y);
                }
            } else {
                for (int k = 0; k < WT; ++k) {
                    const float2 r = wsum[buf][k * W + cl + q];
                    carry[q] = fmaf(r.x, carry[q], r.y);
                    if (k + 1 == wt) h[q] = carry[q];
                }
            }
        }
        if (a.carry && wt == 0 && live && j < tiles)
#pragma unroll
            for (int q = 0; q < V; ++q) a.carry[(b * tiles + j) * a.C + c + q] = h[q];
        TIO* y = static_cast<TIO*>(a.y) + at;
#pragma unroll
        for (int s = 0; s < kLC; ++s) {
#pragma unroll
            for (int q = 0; q < V; ++q) h[q] = gate_step(sg[s][q], h[q], x[s][q]);
            if (s < n) Vec<TIO, V>::store(y + s * a.C, h);
        }
    }
    if (a.state_out && rank == 0 && wt == 0 && live)
#pragma unroll
        for (int q = 0; q < V; ++q) a.state_out[b * a.C + c + q] = carry[q];
}

// Gradients, in reverse time.  With m_t the gradient reaching h_t from the later tokens
// (m_{T-1} = gstate) and lam_t = gy_t + m_t:
//   gx_t = i_t lam_t,  gg_t = f_t i_t (h_{t-1} - x_t) lam_t,  m_{t-1} = f_t lam_t
// A span maps m by m_out = A m_in + M with the forward's A, so the split over warps, blocks and
// strides is the forward's mirrored.  h_{t-1} comes from the tile's saved entering state and the
// forward recurrence of the tile's own steps (the warps' H, exchanged together with M): g, x and
// gy are read once and no other per-token value is needed.
template <typename TIO, int V>
__global__ void __launch_bounds__(kThreads) scan_bwd(ScanArgs a) {
    __shared__ float wa[2][kNW * 32 * V], wh[2][kNW * 32 * V], wm[2][kNW * 32 * V];
    __shared__ float2 csum[2][kMaxCluster][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int WT = 1 << a.wt_log, wt = warp & (WT - 1), wc = warp >> a.wt_log;
    const int W = (kNW >> a.wt_log) * 32 * V;
    const int cl = (wc * 32 + lane) * V;
    const uint32_t S = cluster_size(), rank = cluster_rank();
    const int64_t unit = blockIdx.x / S, b = unit / a.groups;
    const int64_t c = (unit % a.groups) * W + cl;
    const bool live = c < a.C;
    const int64_t tile = (int64_t)WT * kLC, tiles = (a.T + tile - 1) / tile;
    grid_dep_launch_dependents();
    if (S > 1) cluster_arrive();
    grid_dep_wait();  // before any global memory access
    float carry[V];
#pragma unroll
    for (int q = 0; q < V; ++q) carry[q] = live && a.gstate ? a.gstate[b * a.C + c + q] : 0.f;
    if (S > 1) cluster_wait();

    int buf = 0;
    for (int64_t j0 = 0; j0 < tiles; j0 += S, buf ^= 1) {
        const int64_t j = tiles - 1 - j0 - rank;  // < 0: past the sequence's start
        const int64_t t0 = j * tile + wt * kLC;
        const int n = live && j >= 0 && t0 < a.T ? (int)min64(kLC, a.T - t0) : 0;
        const int64_t at = (b * a.T + t0) * a.C + c;
        float sg[kLC][V], x[kLC][V], gy[kLC][V], h[V];
        load_rows<TIO, V>(static_cast<const TIO*>(a.g) + at, a.C, n, INFINITY, sg);
        load_rows<TIO, V>(static_cast<const TIO*>(a.x) + at, a.C, n, 0.f, x);
        load_rows<TIO, V>(static_cast<const TIO*>(a.gy) + at, a.C, n, 0.f, gy);
#pragma unroll
        for (int q = 0; q < V; ++q) h[q] = live && j >= 0 ? a.carry[(b * tiles + j) * a.C + c + q] : 0.f;
        float A[V], H[V], M[V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
            A[q] = 1.f;
            H[q] = 0.f;
            M[q] = 0.f;
        }
#pragma unroll
        for (int s = 0; s < kLC; ++s)
#pragma unroll
            for (int q = 0; q < V; ++q) {
                sg[s][q] = signed_gate(sg[s][q]);
                A[q] = gate_decay(sg[s][q], A[q]);
                H[q] = gate_step(sg[s][q], H[q], x[s][q]);
            }
#pragma unroll
        for (int s = kLC - 1; s >= 0; --s)
#pragma unroll
            for (int q = 0; q < V; ++q) M[q] = gate_decay(sg[s][q], gy[s][q] + M[q]);
#pragma unroll
        for (int q = 0; q < V; ++q) {
            wa[buf][wt * W + cl + q] = A[q];
            wh[buf][wt * W + cl + q] = H[q];
            wm[buf][wt * W + cl + q] = M[q];
        }
        __syncthreads();
        if (S > 1) {
            if (wt == 0) {
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    float2 tot = make_float2(1.f, 0.f);
                    for (int k = WT - 1; k >= 0; --k) {
                        const float ak = wa[buf][k * W + cl + q];
                        tot = make_float2(tot.x * ak, fmaf(ak, tot.y, wm[buf][k * W + cl + q]));
                    }
                    const uint32_t at_s = smem_u32(&csum[buf][rank][cl + q]);
                    for (uint32_t k = 0; k < S; ++k) st_cluster_f2(at_s, k, tot);
                }
            }
            cluster_arrive();
            cluster_wait();
        }
        float m[V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
            for (int k = 0; k < wt; ++k) h[q] = fmaf(wa[buf][k * W + cl + q], h[q], wh[buf][k * W + cl + q]);
            m[q] = carry[q];
            if (S > 1) {
                for (uint32_t k = 0; k < S; ++k) {
                    const float2 r = csum[buf][k][cl + q];
                    carry[q] = fmaf(r.x, carry[q], r.y);
                    if (k + 1 == rank) m[q] = carry[q];
                }
                for (int k = WT - 1; k > wt; --k) m[q] = fmaf(wa[buf][k * W + cl + q], m[q], wm[buf][k * W + cl + q]);
            } else {
                for (int k = WT - 1; k >= 0; --k) {
                    carry[q] = fmaf(wa[buf][k * W + cl + q], carry[q], wm[buf][k * W + cl + q]);
                    if (k - 1 == wt) m[q] = carry[q];
                }
            }
        }
#pragma unroll
        for (int s = 0; s < kLC; ++s)
#pragma unroll
            for (int q = 0; q < V; ++q) {  // x becomes f i (h_{t-1} - x_t); f i = |s| (1 - |s|)
                const float before = h[q], small = fabsf(sg[s][q]);
                h[q] = gate_step(sg[s][q], before, x[s][q]);
                x[s][q] = fmaf(-small, small, small) * (before - x[s][q]);
            }
        TIO* gx = static_cast<TIO*>(a.y) + at;
        TIO* gg = static_cast<TIO*>(a.gg) + at;
#pragma unroll
        for (int s = kLC - 1; s >= 0; --s) {
            float ox[V], og[V];
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float lam = gy[s][q] + m[q];
                ox[q] = gate_input(sg[s][q], lam);
                og[q] = x[s][q] * lam;
                m[q] = gate_decay(sg[s][q], lam);
            }
            if (s < n) {
                Vec<TIO, V>::store(gx + s * a.C, ox);
                Vec<TIO, V>::store(gg + s * a.C, og);
            }
        }
    }
    if (a.state_out && rank == 0 && wt == 0 && live)
#pragma unroll
        for (int q = 0; q < V; ++q) a.state_out[b * a.C + c + q] = carry[q];
}

// One token per row-channel: h <- f h + i x, y = h.  Bound by the bytes of g, x, y and the
// state in and out.
template <typename TIO, int V>
__global__ void __launch_bounds__(256) step_kernel(int64_t n, const TIO* __restrict__ g, const TIO* __restrict__ x,
                                                   float* __restrict__ state, TIO* __restrict__ y) {
    grid_dep_launch_dependents();
    grid_dep_wait();  // before any global memory access
    const int64_t stride = (int64_t)gridDim.x * blockDim.x * V;
    for (int64_t k = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * V; k < n; k += stride) {
        float gv[V], xv[V], h[V];
        Vec<TIO, V>::load(g + k, gv);
        Vec<TIO, V>::load(x + k, xv);
        Vec<float, V>::load(state + k, h);
#pragma unroll
        for (int q = 0; q < V; ++q) h[q] = gate_step(signed_gate(gv[q]), h[q], xv[q]);
        Vec<float, V>::store(state + k, h);
        Vec<TIO, V>::store(y + k, h);
    }
}

__global__ void copy_or_zero(int64_t n, const float* in, float* out) {
    grid_dep_launch_dependents();
    grid_dep_wait();  // before any global memory access
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
        out[i] = in ? in[i] : 0.f;
}

struct ScanGeom {
    int wt_log, S;
    int64_t groups, blocks;
};

int sm_count() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

ScanGeom scan_geometry(const GatedScanShape& s, int V) {
    ScanGeom g;
    g.wt_log = 0;
    while ((1 << g.wt_log) < kNW && (int64_t)(kLC << g.wt_log) < s.T) ++g.wt_log;
    const int64_t W = (int64_t)(kNW >> g.wt_log) * 32 * V;
    g.groups = (s.C + W - 1) / W;
    const int64_t units = s.B * g.groups, tiles = (s.T + kTile - 1) / kTile;
    g.S = 1;
    while (g.S < kMaxCluster && g.S < tiles && units * g.S < 2 * sm_count()) g.S *= 2;
    g.blocks = units * g.S;
    return g;
}

template <typename... KArgs>
cudaError_t launch_cluster(void (*kern)(KArgs...), const ScanGeom& g, const ScanArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)g.blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = kProgrammaticLaunch ? 1 : 0;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim = {(unsigned)g.S, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename TIO, int V>
cudaError_t launch_scan(const GatedScanShape& s, ScanArgs a, bool backward, cudaStream_t stream) {
    const ScanGeom g = scan_geometry(s, V);
    a.groups = g.groups;
    a.wt_log = g.wt_log;
    return launch_cluster(backward ? scan_bwd<TIO, V> : scan_fwd<TIO, V>, g, a, stream);
}

// channels per lane: bf16 pairs where every row starts on a pair (two channels fill a 32-bit
// access), single channels otherwise
cudaError_t dispatch_scan(const GatedScanShape& s, const ScanArgs& a, bool backward, cudaStream_t stream) {
    if (s.io == 0) return launch_scan<float, 1>(s, a, backward, stream);
    if (s.C % 2 == 0) return launch_scan<__nv_bfloat16, 2>(s, a, backward, stream);
    return launch_scan<__nv_bfloat16, 1>(s, a, backward, stream);
}

unsigned flat_blocks(int64_t units) {
    const int64_t b = (units + 255) / 256, cap = (int64_t)sm_count() * 8;
    return (unsigned)(b < cap ? b : cap);
}

}  // namespace

bool gated_scan_fits(const GatedScanShape& s) {
    // the most blocks any split takes: every 32 channels of every sequence, kMaxCluster deep
    return s.B <= INT32_MAX / kMaxCluster / ((s.C + 31) / 32);
}

cudaError_t launch_gated_scan_forward(const GatedScanShape& s, const void* g, const void* x, const float* state_in,
                                      void* y, float* state_out, float* carry, cudaStream_t stream) {
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
    return dispatch_scan(s, a, false, stream);
}

cudaError_t launch_gated_scan_backward(const GatedScanShape& s, const void* g, const void* x, const float* carry,
                                       const void* gy, const float* gstate_out, void* gg, void* gx, float* gstate_in,
                                       cudaStream_t stream) {
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
    return dispatch_scan(s, a, true, stream);
}

cudaError_t launch_gated_scan_step(int64_t n, int io, const void* g, const void* x, float* state, void* y,
                                   cudaStream_t s) {
    if (io == 1) {
        const __nv_bfloat16 *gg = static_cast<const __nv_bfloat16*>(g), *xx = static_cast<const __nv_bfloat16*>(x);
        __nv_bfloat16* yy = static_cast<__nv_bfloat16*>(y);
        if (n % 4 == 0)
            return launch_pdl(step_kernel<__nv_bfloat16, 4>, dim3(flat_blocks(n / 4)), dim3(256), 0, s, n, gg, xx, state, yy);
        return launch_pdl(step_kernel<__nv_bfloat16, 1>, dim3(flat_blocks(n)), dim3(256), 0, s, n, gg, xx, state, yy);
    }
    const float *gg = static_cast<const float*>(g), *xx = static_cast<const float*>(x);
    float* yy = static_cast<float*>(y);
    if (n % 4 == 0)
        return launch_pdl(step_kernel<float, 4>, dim3(flat_blocks(n / 4)), dim3(256), 0, s, n, gg, xx, state, yy);
    return launch_pdl(step_kernel<float, 1>, dim3(flat_blocks(n)), dim3(256), 0, s, n, gg, xx, state, yy);
}

}  // namespace wkvb
