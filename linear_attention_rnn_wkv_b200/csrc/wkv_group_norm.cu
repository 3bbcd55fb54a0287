// Gated group norm over the channels of each row (declarations and contract in include/wkv.h):
//   n = (x - mean) / sqrt(var + eps) per row and group of D channels,  a = n weight + bias
//   y = a act(z),  or act(a) without z
// and its gradients (r = 1 / sqrt(var + eps)):
//   ga = gy act(z), gz = gy a act'(z)   |   ga = gy act'(a)
//   gbias = sum over rows of ga,  gweight = sum over rows of ga n,  gn = ga weight
//   gx = r (gn - mean gn - n mean(gn n))
// The backward reads x anyway, so it takes the statistics again instead of having them stored.
//
// A group's row is held in registers by a team of LPG lanes (up to NV vectors of V channels per
// lane): every tensor is read once and written once.  The variance is the mean of squared
// differences from the mean, in a second pass over the registers.  A team keeps its group and
// walks the rows, so weight, bias and the sums of their gradients stay in registers.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "wkv_device.cuh"
#include "wkv_gated_internal.h"
#include "wkv_internal.h"
#include "wkv_vec.cuh"

namespace wkvb {
namespace {

constexpr int kTeamWarps = 4;    // warps per block, each on its own rows
constexpr int kWide = 256;       // threads of a block that takes a whole group

struct NormArgs {
    int64_t rows, C;
    int G, D;
    float eps;
    int act;
    const void *x, *z, *gy;
    const float *weight, *bias;
    void *y;         // forward: y; backward: gx
    void *gz;
    float* part;     // backward: [2][gridDim.y][C] sums of gweight, gbias, or null
};

// sigma(v) and 1 - sigma(v), each relatively accurate
__device__ __forceinline__ void logistic(float v, float& p, float& q) {
    const float e = ex2(-fabsf(v) * kLog2e), r = rcp(1.f + e), small = e * r;
    p = v >= 0.f ? r : small;
    q = v >= 0.f ? small : r;
}
__device__ __forceinline__ float act_value(int act, float v) {
    if (act == kActNone) return v;
    float p, q;
    logistic(v, p, q);
    return act == kActSilu ? v * p : p;
}
// act(v), and its derivative in d
__device__ __forceinline__ float act_slope(int act, float v, float& d) {
    if (act == kActNone) {
        d = 1.f;
        return v;
    }
    float p, q;
    logistic(v, p, q);
    if (act == kActSilu) {
        d = fmaf(v * p, q, p);
        return v * p;
    }
    d = p * q;
    return p;
}

template <int LPG>
__device__ __forceinline__ float team_sum(float v) {
#pragma unroll
    for (int o = LPG / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename TIO, int V>
__device__ __forceinline__ void load_or(bool ok, const TIO* p, float other, float (&o)[V]) {
    if (ok) {
        Vec<TIO, V>::load(p, o);
    } else {
#pragma unroll
        for (int q = 0; q < V; ++q) o[q] = other;
    }
}
template <int V>
__device__ __forceinline__ void load_param(bool ok, const float* p, int64_t at, float other, float (&o)[V]) {
#pragma unroll
    for (int q = 0; q < V; ++q) o[q] = ok && p ? p[at + q] : other;
}

// The lanes of one team and what they hold of a row: normalised values n (zero past the group).
template <int V, int LPG, int NV>
struct Team {
    int64_t col[NV];  // first channel of each vector
    bool ok[NV];
    bool live;

    __device__ __forceinline__ Team(const NormArgs& a) {
        const int lane = threadIdx.x & 31;
        const int64_t g = (int64_t)blockIdx.x * (32 / LPG) + lane / LPG;
        live = g < a.G;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = (lane % LPG + i * LPG) * V;
            ok[i] = live && at < a.D;
            col[i] = g * a.D + at;
        }
    }
    // x -> n, returns r
    __device__ __forceinline__ float normalise(const NormArgs& a, float inv, float (&x)[NV][V]) const {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q) s += x[i][q];
        const float mean = team_sum<LPG>(s) * inv;
        s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q) {
                x[i][q] = ok[i] ? x[i][q] - mean : 0.f;
                s = fmaf(x[i][q], x[i][q], s);
            }
        const float r = rsqrtf(fmaf(team_sum<LPG>(s), inv, a.eps));
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q) x[i][q] *= r;
        return r;
    }
};

template <typename TIO, int V, int LPG, int NV>
__global__ void __launch_bounds__(32 * kTeamWarps) norm_fwd(NormArgs a) {
    const Team<V, LPG, NV> t(a);
    const TIO *x = static_cast<const TIO*>(a.x), *z = static_cast<const TIO*>(a.z);
    TIO* y = static_cast<TIO*>(a.y);
    const float inv = 1.f / (float)a.D;
    grid_dep_launch_dependents();
    grid_dep_wait();  // before any global memory access
    float w[NV][V], b[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        load_param<V>(t.ok[i], a.weight, t.col[i], 1.f, w[i]);
        load_param<V>(t.ok[i], a.bias, t.col[i], 0.f, b[i]);
    }
    for (int64_t row = (int64_t)blockIdx.y * kTeamWarps + (threadIdx.x >> 5); row < a.rows;
         row += (int64_t)gridDim.y * kTeamWarps) {
        float n[NV][V], u[NV][V];
#pragma unroll
        for (int i = 0; i < NV; ++i) load_or<TIO, V>(t.ok[i], x + row * a.C + t.col[i], 0.f, n[i]);
        if (z)
#pragma unroll
            for (int i = 0; i < NV; ++i) load_or<TIO, V>(t.ok[i], z + row * a.C + t.col[i], 0.f, u[i]);
        t.normalise(a, inv, n);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float v = fmaf(n[i][q], w[i][q], b[i][q]);
                n[i][q] = z ? v * act_value(a.act, u[i][q]) : act_value(a.act, v);
            }
            if (t.ok[i]) Vec<TIO, V>::store(y + row * a.C + t.col[i], n[i]);
        }
    }
}

template <typename TIO, int V, int LPG, int NV>
__global__ void __launch_bounds__(32 * kTeamWarps) norm_bwd(NormArgs a) {
    const Team<V, LPG, NV> t(a);
    const TIO *x = static_cast<const TIO*>(a.x), *z = static_cast<const TIO*>(a.z), *gy = static_cast<const TIO*>(a.gy);
    TIO *gx = static_cast<TIO*>(a.y), *gz = static_cast<TIO*>(a.gz);
    const float inv = 1.f / (float)a.D;
    grid_dep_launch_dependents();
    grid_dep_wait();  // before any global memory access
    float w[NV][V], b[NV][V], gw[NV][V], gb[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        load_param<V>(t.ok[i], a.weight, t.col[i], 1.f, w[i]);
        load_param<V>(t.ok[i], a.bias, t.col[i], 0.f, b[i]);
#pragma unroll
        for (int q = 0; q < V; ++q) gw[i][q] = gb[i][q] = 0.f;
    }
    for (int64_t row = (int64_t)blockIdx.y * kTeamWarps + (threadIdx.x >> 5); row < a.rows;
         row += (int64_t)gridDim.y * kTeamWarps) {
        float n[NV][V], u[NV][V], g[NV][V];
#pragma unroll
        for (int i = 0; i < NV; ++i) load_or<TIO, V>(t.ok[i], x + row * a.C + t.col[i], 0.f, n[i]);
        if (z)
#pragma unroll
            for (int i = 0; i < NV; ++i) load_or<TIO, V>(t.ok[i], z + row * a.C + t.col[i], 0.f, u[i]);
#pragma unroll
        for (int i = 0; i < NV; ++i) load_or<TIO, V>(t.ok[i], gy + row * a.C + t.col[i], 0.f, g[i]);
        const float r = t.normalise(a, inv, n);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float v = fmaf(n[i][q], w[i][q], b[i][q]);
                float d;
                if (z) {
                    const float act = act_slope(a.act, u[i][q], d);
                    u[i][q] = g[i][q] * v * d;  // gz
                    g[i][q] *= act;
                } else {
                    act_slope(a.act, v, d);
                    g[i][q] *= d;
                }
                gb[i][q] += g[i][q];
                gw[i][q] = fmaf(g[i][q], n[i][q], gw[i][q]);
                g[i][q] *= w[i][q];  // gn
                s1 += g[i][q];
                s2 = fmaf(g[i][q], n[i][q], s2);
            }
        s1 = team_sum<LPG>(s1) * inv;
        s2 = team_sum<LPG>(s2) * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int q = 0; q < V; ++q) g[i][q] = r * (g[i][q] - fmaf(n[i][q], s2, s1));
            if (t.ok[i]) {
                Vec<TIO, V>::store(gx + row * a.C + t.col[i], g[i]);
                if (z) Vec<TIO, V>::store(gz + row * a.C + t.col[i], u[i]);
            }
        }
    }
    if (!a.part) return;
    // the block's sums, its warps in order
    __shared__ float sums[kTeamWarps][32 * NV * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q) sums[warp][(i * V + q) * 32 + lane] = which ? gb[i][q] : gw[i][q];
        __syncthreads();
        if (warp == 0)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    float s = 0.f;
#pragma unroll
                    for (int k = 0; k < kTeamWarps; ++k) s += sums[k][(i * V + q) * 32 + lane];
                    if (t.ok[i]) a.part[((int64_t)which * gridDim.y + blockIdx.y) * a.C + t.col[i] + q] = s;
                }
    }
}

// Groups of more than 128 vectors: a block per group, the row read again for each pass (from the
// caches: a row's group is at most a few tens of KB), any D.
__device__ __forceinline__ float block_sum(float v, float* buf) {
    v = team_sum<32>(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kWide / 32; ++k) s += buf[k];
    return s;
}

template <typename TIO, int V, bool BWD>
__global__ void __launch_bounds__(kWide) norm_wide(NormArgs a) {
    __shared__ float buf[kWide / 32];
    const int64_t col = (int64_t)blockIdx.x * a.D;
    const TIO *x = static_cast<const TIO*>(a.x), *z = static_cast<const TIO*>(a.z), *gy = static_cast<const TIO*>(a.gy);
    TIO *y = static_cast<TIO*>(a.y), *gz = static_cast<TIO*>(a.gz);
    const float inv = 1.f / (float)a.D;
    grid_dep_launch_dependents();
    grid_dep_wait();  // before any global memory access
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const int64_t at = row * a.C + col;
        float s = 0.f;
        for (int64_t c = (int64_t)threadIdx.x * V; c < a.D; c += kWide * V) {
            float v[V];
            Vec<TIO, V>::load(x + at + c, v);
#pragma unroll
            for (int q = 0; q < V; ++q) s += v[q];
        }
        const float mean = block_sum(s, buf) * inv;
        s = 0.f;
        for (int64_t c = (int64_t)threadIdx.x * V; c < a.D; c += kWide * V) {
            float v[V];
            Vec<TIO, V>::load(x + at + c, v);
#pragma unroll
            for (int q = 0; q < V; ++q) s = fmaf(v[q] - mean, v[q] - mean, s);
        }
        const float r = rsqrtf(fmaf(block_sum(s, buf), inv, a.eps));
        if constexpr (!BWD) {
            for (int64_t c = (int64_t)threadIdx.x * V; c < a.D; c += kWide * V) {
                float v[V], u[V], w[V], b[V];
                Vec<TIO, V>::load(x + at + c, v);
                if (z) Vec<TIO, V>::load(z + at + c, u);
                load_param<V>(true, a.weight, col + c, 1.f, w);
                load_param<V>(true, a.bias, col + c, 0.f, b);
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float t = fmaf((v[q] - mean) * r, w[q], b[q]);
                    v[q] = z ? t * act_value(a.act, u[q]) : act_value(a.act, t);
                }
                Vec<TIO, V>::store(y + at + c, v);
            }
        } else {
            float s1 = 0.f, s2 = 0.f;
            const bool first = row == blockIdx.y;
            // two passes over the gradients: their sums, then the results
            for (int pass = 0; pass < 2; ++pass) {
                for (int64_t c = (int64_t)threadIdx.x * V; c < a.D; c += kWide * V) {
                    float v[V], u[V], g[V], w[V], b[V];
                    Vec<TIO, V>::load(x + at + c, v);
                    if (z) Vec<TIO, V>::load(z + at + c, u);
                    Vec<TIO, V>::load(gy + at + c, g);
                    load_param<V>(true, a.weight, col + c, 1.f, w);
                    load_param<V>(true, a.bias, col + c, 0.f, b);
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        const float n = (v[q] - mean) * r, t = fmaf(n, w[q], b[q]);
                        float d;
                        if (z) {
                            const float act = act_slope(a.act, u[q], d);
                            u[q] = g[q] * t * d;
                            g[q] *= act;
                        } else {
                            act_slope(a.act, t, d);
                            g[q] *= d;
                        }
                        if (pass == 0) {
                            s1 = fmaf(g[q], w[q], s1);
                            s2 = fmaf(g[q] * w[q], n, s2);
                            if (a.part) {  // this thread's own columns
                                float* pw = a.part + (int64_t)blockIdx.y * a.C + col + c + q;
                                float* pb = pw + (int64_t)gridDim.y * a.C;
                                *pw = fmaf(g[q], n, first ? 0.f : *pw);
                                *pb = g[q] + (first ? 0.f : *pb);
                            }
                        } else {
                            v[q] = r * (g[q] * w[q] - fmaf(n, s2, s1));
                        }
                    }
                    if (pass == 1) {
                        Vec<TIO, V>::store(y + at + c, v);
                        if (z) Vec<TIO, V>::store(gz + at + c, u);
                    }
                }
                if (pass == 0) {
                    s1 = block_sum(s1, buf) * inv;
                    s2 = block_sum(s2, buf) * inv;
                }
            }
        }
    }
}

// gweight and gbias: the blocks' sums, in a fixed order (eight interleaved partial sums)
constexpr int kReduceRows = 8;
__global__ void __launch_bounds__(32 * kReduceRows) norm_reduce(int64_t C, int parts, const float* part, float* gw, float* gb) {
    __shared__ float sums[kReduceRows][33];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float* out = blockIdx.y ? gb : gw;
    grid_dep_launch_dependents();
    grid_dep_wait();  // before any global memory access
    float s = 0.f;
    if (c < C)
        for (int k = slice; k < parts; k += kReduceRows) s += part[((int64_t)blockIdx.y * parts + k) * C + c];
    sums[slice][lane] = s;
    __syncthreads();
    if (slice == 0 && c < C && out) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < kReduceRows; ++k) s += sums[k][lane];
        out[c] = s;
    }
}

// no rows: zero gradients
__global__ void norm_zero(int64_t C, float* gw, float* gb) {
    grid_dep_launch_dependents();
    grid_dep_wait();  // before any global memory access
    for (int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; c < C; c += (int64_t)gridDim.x * blockDim.x) {
        if (gw) gw[c] = 0.f;
        if (gb) gb[c] = 0.f;
    }
}

// How a group is laid over lanes: V channels per vector, LPG lanes, NV vectors per lane; LPG = 0:
// a block per group.  The fewest lanes that hold it, so that a warp covers as many groups as it can.
struct NormPlan {
    int V, LPG, NV;
    int64_t x;  // blocks along the groups
    int y;      // blocks along the rows
};

constexpr int kBlocksFwd = 148 * 12, kBlocksBwd = 148 * 6, kBlocksWide = 148 * 8;

NormPlan norm_plan(const GroupNormShape& s, bool backward) {
    const int64_t D = s.C / s.groups;
    const int full = s.io == 1 ? 8 : 4;
    NormPlan p;
    p.V = D % full == 0 ? full : (s.io == 1 && D % 2 == 0 ? 2 : 1);
    const int64_t nvec = D / p.V;
    p.NV = nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4;
    p.LPG = nvec <= 4 ? 4 : nvec <= 8 ? 8 : nvec <= 16 ? 16 : 32;
    if (nvec > 128) p.LPG = 0;
    int64_t most;
    if (p.LPG) {
        p.x = (s.groups + 32 / p.LPG - 1) / (32 / p.LPG);
        most = (s.rows + kTeamWarps - 1) / kTeamWarps;
    } else {
        p.x = s.groups;
        most = s.rows;
    }
    int64_t y = (p.LPG ? (backward ? kBlocksBwd : kBlocksFwd) : kBlocksWide) / p.x;
    if (y < 1) y = 1;
    p.y = (int)(y < most ? y : most);
    return p;
}

template <typename TIO, int V, int LPG, int NV>
cudaError_t launch_team(const NormPlan& p, const NormArgs& a, bool backward, cudaStream_t s) {
    return launch_pdl(backward ? norm_bwd<TIO, V, LPG, NV> : norm_fwd<TIO, V, LPG, NV>, dim3((unsigned)p.x, (unsigned)p.y),
                      dim3(32 * kTeamWarps), 0, s, a);
}

template <typename TIO, int V>
cudaError_t launch_norm(const NormPlan& p, const NormArgs& a, bool backward, cudaStream_t s) {
    if (p.LPG == 0)
        return launch_pdl(backward ? norm_wide<TIO, V, true> : norm_wide<TIO, V, false>, dim3((unsigned)p.x, (unsigned)p.y),
                          dim3(kWide), 0, s, a);
    if (p.LPG == 4) return launch_team<TIO, V, 4, 1>(p, a, backward, s);
    if (p.LPG == 8) return launch_team<TIO, V, 8, 1>(p, a, backward, s);
    if (p.LPG == 16) return launch_team<TIO, V, 16, 1>(p, a, backward, s);
    if (p.NV == 1) return launch_team<TIO, V, 32, 1>(p, a, backward, s);
    if (p.NV == 2) return launch_team<TIO, V, 32, 2>(p, a, backward, s);
    return launch_team<TIO, V, 32, 4>(p, a, backward, s);
}

cudaError_t launch_norm(const GroupNormShape& s, const NormPlan& p, const NormArgs& a, bool backward, cudaStream_t stream) {
    if (s.io == 0)
        return p.V == 4 ? launch_norm<float, 4>(p, a, backward, stream) : launch_norm<float, 1>(p, a, backward, stream);
    if (p.V == 8) return launch_norm<__nv_bfloat16, 8>(p, a, backward, stream);
    if (p.V == 2) return launch_norm<__nv_bfloat16, 2>(p, a, backward, stream);
    return launch_norm<__nv_bfloat16, 1>(p, a, backward, stream);
}

NormArgs norm_args(const GroupNormShape& s, const void* x, const void* z, const float* weight, const float* bias) {
    NormArgs a = {};
    a.rows = s.rows;
    a.C = s.C;
    a.G = (int)s.groups;
    a.D = (int)(s.C / s.groups);
    a.eps = s.eps;
    a.act = s.act;
    a.x = x;
    a.z = z;
    a.weight = weight;
    a.bias = bias;
    return a;
}

}  // namespace

size_t group_norm_workspace_bytes(const GroupNormShape& s) {
    return (size_t)2 * (size_t)norm_plan(s, true).y * (size_t)s.C * sizeof(float);
}

cudaError_t launch_group_norm_forward(const GroupNormShape& s, const void* x, const void* z, const float* weight,
                                      const float* bias, void* y, cudaStream_t stream) {
    NormArgs a = norm_args(s, x, z, weight, bias);
    a.y = y;
    return launch_norm(s, norm_plan(s, false), a, false, stream);
}

cudaError_t launch_group_norm_backward(const GroupNormShape& s, const void* x, const void* z, const float* weight,
                                       const float* bias, const void* gy, void* gx, void* gz, float* gweight, float* gbias,
                                       void* workspace, cudaStream_t stream) {
    if (s.rows == 0)
        return launch_pdl(norm_zero, dim3((unsigned)((s.C + 255) / 256)), dim3(256), 0, stream, s.C, gweight, gbias);
    NormArgs a = norm_args(s, x, z, weight, bias);
    a.gy = gy;
    a.y = gx;
    a.gz = gz;
    a.part = gweight || gbias ? static_cast<float*>(workspace) : nullptr;
    const NormPlan p = norm_plan(s, true);
    cudaError_t e = launch_norm(s, p, a, true, stream);
    if (e == cudaSuccess && a.part)
        e = launch_pdl(norm_reduce, dim3((unsigned)((s.C + 31) / 32), 2), dim3(32 * kReduceRows), 0, stream, s.C, p.y, (const float*)a.part,
                       gweight, gbias);
    return e;
}

}  // namespace wkvb
