// Gated group norm over the channels of each row (declarations and contract in include/wkv.h):
//   n = (x - mean) / sqrt(var + eps) per row and group of D channels,  a = n weight + bias
//   y = a act(z),  or act(a) without z
// and its gradients (r = 1 / sqrt(var + eps)):
//   ga = gy act(z), gz = gy a act'(z)   |   ga = gy act'(a)
//   gbias = sum over rows of ga,  gweight = sum over rows of ga n,  gn = ga weight
//   gx = r (gn - mean gn - n mean(gn n))
// The backward reads x anyway, so it takes the statistics again instead of having them stored.
//
// A group's row is held in registers by a team of LPG lanes (NV vectors of V channels per lane;
// teams of 4 to 32 lanes within a warp, or a block of 128 to 512 threads): every tensor is read
// once and written once.  The variance is the mean of squared differences from the mean, in a
// second pass over the registers.  A team keeps its group and walks the rows, so weight, bias and
// the sums of their gradients stay in registers, and the next row's vectors are under way while
// one is computed.  Two channels share an instruction (packed fp32): in bf16 the instructions,
// not the bytes, were the limit.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "wkv_device.cuh"
#include "wkv_gated_internal.h"
#include "wkv_internal.h"
#include "wkv_vec.cuh"

namespace wkvb {
namespace {

constexpr int kTeamWarps = 4;  // warps per block of teams within a warp, each on its own rows
constexpr int kWide = 256;     // threads of a block that reads its group again for each pass

// Blocks of 128 threads resident per SM, by the channels a thread holds (its registers): the
// rows are walked by exactly one such wave.  16384 x 2048 in 32 groups, bf16, forward with 6, 8, 12
// blocks per SM 40.9, 35.4, 40.3 us (8 fit), backward with 4, 5, 6 71.4, 63.3, 83.2 us (5 fit).
constexpr int team_threads(int LPG) { return LPG <= 32 ? 32 * kTeamWarps : LPG; }
constexpr int resident(int held, int threads, bool backward) {
    const int r = backward ? (held <= 2 ? 10 : held <= 4 ? 6 : held <= 8 ? 5 : 3)
                           : (held <= 2 ? 16 : held <= 4 ? 10 : held <= 8 ? 8 : 4);
    return r * 128 / threads > 0 ? r * 128 / threads : 1;
}

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

// ---- pairs of channels ----
__device__ __forceinline__ float2 all2(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
// sigma: 2^(-v log2 e) = inf gives 0
__device__ __forceinline__ float2 logistic2(float2 v) {
    const float2 t = mul2(v, all2(-kLog2e)), d = add2(make_float2(ex2(t.x), ex2(t.y)), all2(1.f));
    return make_float2(rcp(d.x), rcp(d.y));
}
__device__ __forceinline__ float2 act_value2(int act, float2 v) {
    if (act == kActNone) return v;
    const float2 p = logistic2(v);
    return act == kActSilu ? mul2(v, p) : p;
}
// SiLU' = p + v p (1 - p): the rounding of 1 - p, at most 2^-24, enters times |v| p.  sigma' = p (1 - p)
// needs 1 - p relatively accurate where p is near 1.
__device__ __forceinline__ float2 act_slope2(int act, float2 v, float2& d) {
    if (act == kActSilu) {
        const float2 p = logistic2(v), vp = mul2(v, p);
        d = fma2(vp, fma2(p, all2(-1.f), all2(1.f)), p);
        return vp;
    }
    float2 r;
    r.x = act_slope(act, v.x, d.x);
    r.y = act_slope(act, v.y, d.y);
    return r;
}

// V adjacent channels as loaded, and as (V + 1) / 2 pairs (a single channel: the pair's x, y = 0)
template <typename TIO, int V>
struct Raw;
template <>
struct Raw<float, 4> {
    using R = float4;
    static __device__ __forceinline__ void unpack(R r, float2 (&o)[2]) {
        o[0] = make_float2(r.x, r.y);
        o[1] = make_float2(r.z, r.w);
    }
    static __device__ __forceinline__ R pack(const float2 (&o)[2]) { return make_float4(o[0].x, o[0].y, o[1].x, o[1].y); }
};
template <>
struct Raw<float, 1> {
    using R = float;
    static __device__ __forceinline__ void unpack(R r, float2 (&o)[1]) { o[0] = make_float2(r, 0.f); }
    static __device__ __forceinline__ R pack(const float2 (&o)[1]) { return o[0].x; }
};
template <>
struct Raw<__nv_bfloat16, 8> {
    using R = uint4;
    static __device__ __forceinline__ void unpack(R r, float2 (&o)[4]) {
        o[0] = make_float2(bf_lo(r.x), bf_hi(r.x));
        o[1] = make_float2(bf_lo(r.y), bf_hi(r.y));
        o[2] = make_float2(bf_lo(r.z), bf_hi(r.z));
        o[3] = make_float2(bf_lo(r.w), bf_hi(r.w));
    }
    static __device__ __forceinline__ R pack(const float2 (&o)[4]) {
        return make_uint4(bf_pack(o[0].x, o[0].y), bf_pack(o[1].x, o[1].y), bf_pack(o[2].x, o[2].y), bf_pack(o[3].x, o[3].y));
    }
};
template <>
struct Raw<__nv_bfloat16, 2> {
    using R = uint32_t;
    static __device__ __forceinline__ void unpack(R r, float2 (&o)[1]) { o[0] = make_float2(bf_lo(r), bf_hi(r)); }
    static __device__ __forceinline__ R pack(const float2 (&o)[1]) { return bf_pack(o[0].x, o[0].y); }
};
template <>
struct Raw<__nv_bfloat16, 1> {
    using R = uint16_t;
    static __device__ __forceinline__ void unpack(R r, float2 (&o)[1]) { o[0] = make_float2(bf_lo(r), 0.f); }
    static __device__ __forceinline__ R pack(const float2 (&o)[1]) { return (uint16_t)bf_pack(o[0].x, 0.f); }
};

template <int V>
__device__ __forceinline__ void load_param(bool ok, const float* p, int64_t at, float other, float (&o)[V]) {
#pragma unroll
    for (int q = 0; q < V; ++q) o[q] = ok && p ? p[at + q] : other;
}

template <int LPG>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = (LPG < 32 ? LPG : 32) / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The lanes of one team.  ALL: every lane of a team holds NV whole vectors (a team past the last
// group then reads the last group's values again and writes nothing).
template <typename TIO, int V, int LPG, int NV, bool ALL>
struct Team {
    static constexpr int NP = (V + 1) / 2;
    using R = typename Raw<TIO, V>::R;
    const NormArgs& a;
    int64_t col[NV];      // first channel of each vector
    bool ok[NV];          // there is such a vector
    bool live;            // and such a group
    float inv;
    int64_t row, step;    // this team's rows
    float (*buf)[LPG / 32 + 1];  // a block's partial sums (teams of more than a warp): two, in turn
    int turn = 0;

    __device__ __forceinline__ Team(const NormArgs& args, float (*b)[LPG / 32 + 1]) : a(args), buf(b) {
        const int in = LPG <= 32 ? (threadIdx.x & 31) % LPG : threadIdx.x;
        int64_t g = blockIdx.x;
        if (LPG <= 32) g = g * (32 / (LPG <= 32 ? LPG : 32)) + (threadIdx.x & 31) / LPG;
        live = g < a.G;
        if (ALL && !live) g = a.G - 1;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = (in + i * LPG) * V;
            ok[i] = ALL || (live && at < a.D);
            col[i] = g * a.D + at;
        }
        inv = 1.f / (float)a.D;
        row = LPG <= 32 ? (int64_t)blockIdx.y * kTeamWarps + (threadIdx.x >> 5) : blockIdx.y;
        step = (int64_t)gridDim.y * (LPG <= 32 ? kTeamWarps : 1);
    }
    __device__ __forceinline__ bool writes(int i) const { return ALL ? live : ok[i]; }
    __device__ __forceinline__ void fetch(const void* p, int64_t r, R (&o)[NV]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            o[i] = R{};
            if (ok[i]) o[i] = *reinterpret_cast<const R*>(static_cast<const TIO*>(p) + r * a.C + col[i]);
        }
    }
    __device__ __forceinline__ void put(void* p, const float2 (&v)[NV][NP]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (writes(i)) *reinterpret_cast<R*>(static_cast<TIO*>(p) + row * a.C + col[i]) = Raw<TIO, V>::pack(v[i]);
    }
    __device__ __forceinline__ void params(const float* p, float other, float2 (&o)[NV][NP]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float t[V];
            load_param<V>(ok[i], p, col[i], other, t);
#pragma unroll
            for (int j = 0; j < NP; ++j) o[i][j] = make_float2(t[2 * j], 2 * j + 1 < V ? t[V == 1 ? 0 : 2 * j + 1] : 0.f);
        }
    }
    // K sums over the team at once
    template <int K>
    __device__ __forceinline__ void sum(float (&v)[K]) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = warp_sum<LPG>(v[k]);
        if constexpr (LPG > 32) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float* b = buf[2 * turn + k];
                if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v[k];
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k) {
                v[k] = 0.f;
#pragma unroll
                for (int w = 0; w < LPG / 32; ++w) v[k] += buf[2 * turn + k][w];
            }
            turn ^= 1;  // written again only behind the next sum's barrier
        }
    }
    // x -> n, returns r
    __device__ __forceinline__ float normalise(float2 (&x)[NV][NP]) {
        float2 s = all2(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < NP; ++j) s = add2(s, x[i][j]);
        float t[1] = {s.x + s.y};
        sum(t);
        const float2 mean = all2(-t[0] * inv);
        s = all2(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                x[i][j] = add2(x[i][j], mean);
                if (!ALL && !ok[i]) x[i][j] = all2(0.f);
                if (V == 1) x[i][j].y = 0.f;
                s = fma2(x[i][j], x[i][j], s);
            }
        t[0] = s.x + s.y;
        sum(t);
        const float r = rsqrtf(fmaf(t[0], inv, a.eps));
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < NP; ++j) x[i][j] = mul2(x[i][j], all2(r));
        return r;
    }
};

template <typename TIO, int V, int LPG, int NV, bool ALL>
__global__ void __launch_bounds__(team_threads(LPG), resident(NV * V, team_threads(LPG), false)) norm_fwd(NormArgs a) {
    using T = Team<TIO, V, LPG, NV, ALL>;
    constexpr int NP = T::NP;
    __shared__ float buf[4][LPG / 32 + 1];
    T t(a, buf);
    grid_dep_launch_dependents();
    grid_dep_wait();  // before any global memory access
    float2 w[NV][NP], b[NV][NP];
    t.params(a.weight, 1.f, w);
    t.params(a.bias, 0.f, b);
    typename T::R rx[NV], rz[NV];
    if (t.row < a.rows) {
        t.fetch(a.x, t.row, rx);
        if (a.z) t.fetch(a.z, t.row, rz);
    }
    for (; t.row < a.rows; t.row += t.step) {
        float2 n[NV][NP], u[NV][NP];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Raw<TIO, V>::unpack(rx[i], n[i]);
            if (a.z) Raw<TIO, V>::unpack(rz[i], u[i]);
        }
        if (t.row + t.step < a.rows) {
            t.fetch(a.x, t.row + t.step, rx);
            if (a.z) t.fetch(a.z, t.row + t.step, rz);
        }
        t.normalise(n);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const float2 v = fma2(n[i][j], w[i][j], b[i][j]);
                n[i][j] = a.z ? mul2(v, act_value2(a.act, u[i][j])) : act_value2(a.act, v);
            }
        t.put(a.y, n);
    }
}

template <typename TIO, int V, int LPG, int NV, bool ALL>
__global__ void __launch_bounds__(team_threads(LPG), resident(NV * V, team_threads(LPG), true)) norm_bwd(NormArgs a) {
    using T = Team<TIO, V, LPG, NV, ALL>;
    constexpr int NP = T::NP;
    __shared__ float buf[4][LPG / 32 + 1];
    T t(a, buf);
    grid_dep_launch_dependents();
    grid_dep_wait();  // before any global memory access
    float2 w[NV][NP], b[NV][NP], gw[NV][NP], gb[NV][NP];
    t.params(a.weight, 1.f, w);
    t.params(a.bias, 0.f, b);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < NP; ++j) gw[i][j] = gb[i][j] = all2(0.f);
    typename T::R rx[NV], rz[NV], rg[NV];
    if (t.row < a.rows) {
        t.fetch(a.x, t.row, rx);
        if (a.z) t.fetch(a.z, t.row, rz);
        t.fetch(a.gy, t.row, rg);
    }
    for (; t.row < a.rows; t.row += t.step) {
        float2 n[NV][NP], u[NV][NP], g[NV][NP];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Raw<TIO, V>::unpack(rx[i], n[i]);
            if (a.z) Raw<TIO, V>::unpack(rz[i], u[i]);
            Raw<TIO, V>::unpack(rg[i], g[i]);
        }
        if (t.row + t.step < a.rows) {
            t.fetch(a.x, t.row + t.step, rx);
            if (a.z) t.fetch(a.z, t.row + t.step, rz);
            t.fetch(a.gy, t.row + t.step, rg);
        }
        const float r = t.normalise(n);
        float2 s1 = all2(0.f), s2 = all2(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const float2 v = fma2(n[i][j], w[i][j], b[i][j]);
                float2 d;
                if (a.z) {
                    const float2 act = act_slope2(a.act, u[i][j], d);
                    u[i][j] = mul2(mul2(g[i][j], v), d);  // gz
                    g[i][j] = mul2(g[i][j], act);
                } else {
                    act_slope2(a.act, v, d);
                    g[i][j] = mul2(g[i][j], d);
                }
                gb[i][j] = add2(gb[i][j], g[i][j]);
                gw[i][j] = fma2(g[i][j], n[i][j], gw[i][j]);
                g[i][j] = mul2(g[i][j], w[i][j]);  // gn
                s1 = add2(s1, g[i][j]);
                s2 = fma2(g[i][j], n[i][j], s2);
            }
        float m[2] = {s1.x + s1.y, s2.x + s2.y};
        t.sum(m);
        const float2 m1 = all2(-m[0] * t.inv), m2 = all2(-m[1] * t.inv);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < NP; ++j) g[i][j] = mul2(add2(g[i][j], fma2(n[i][j], m2, m1)), all2(r));
        t.put(a.y, g);
        if (a.z) t.put(a.gz, u);
    }
    if (!a.part) return;
    float* part[2] = {a.part + (int64_t)blockIdx.y * a.C, a.part + ((int64_t)gridDim.y + blockIdx.y) * a.C};
    if constexpr (LPG > 32) {  // a thread's channels are its own
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q)
                if (t.writes(i)) {
                    part[0][t.col[i] + q] = q & 1 ? gw[i][q / 2].y : gw[i][q / 2].x;
                    part[1][t.col[i] + q] = q & 1 ? gb[i][q / 2].y : gb[i][q / 2].x;
                }
    } else {  // the block's sums, its warps in order
        __shared__ float sums[kTeamWarps][32 * NV * V];
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float2 v = which ? gb[i][q / 2] : gw[i][q / 2];
                    sums[warp][(i * V + q) * 32 + lane] = q & 1 ? v.y : v.x;
                }
            __syncthreads();
            if (warp == 0)
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        float s = 0.f;
#pragma unroll
                        for (int k = 0; k < kTeamWarps; ++k) s += sums[k][(i * V + q) * 32 + lane];
                        if (t.writes(i)) part[which][t.col[i] + q] = s;
                    }
        }
    }
}

// Groups that no team holds: a block per group, the row read again for each pass (from the
// caches: a row's group is at most a few tens of KB), any D.  Far from the copy rate: 8192 x 5120 in one
// group 116 us forward and 381 backward in fp32 (floor 77 and 128), 113 and 487 in bf16 (38 and 64); the
// backward reads x four times, z and gy twice, and adds the parameters' sums in global memory.
__device__ __forceinline__ float block_sum(float v, float* buf) {
    v = warp_sum<32>(v);
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

// gweight and gbias: the blocks' sums, in a fixed order (kReduceRows interleaved partial sums)
constexpr int kReduceRows = 32;
__global__ void __launch_bounds__(32 * kReduceRows) norm_reduce(int64_t C, int parts, const float* part, float* gw, float* gb) {
    __shared__ float sums[kReduceRows][33];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float* out = blockIdx.y ? gb : gw;
    grid_dep_launch_dependents();
    grid_dep_wait();  // before any global memory access
    const float* p = part + (int64_t)blockIdx.y * parts * C + c;
    float s = 0.f;
    if (c < C && out) {
#pragma unroll 8
        for (int k = slice; k < parts; k += kReduceRows) s += p[k * C];
    }
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
// a block reading its group again.  The fewest lanes (of 4, 8, 16, 32, or a block) that hold it, so that a
// warp covers as many groups as it can (bf16 groups of 8 leave three lanes of four empty, odd ones of 65
// half of 32 lanes' slots); V fills 16 bytes where the groups start on them, else 4 bytes, else one channel.
struct NormPlan {
    int V, LPG, NV;
    bool all;   // whole vectors in every lane
    int64_t x;  // blocks along the groups
    int y;      // blocks along the rows
};

constexpr int kSms = 148;  // of the whole device; on a part of it the grid is only not one even wave

NormPlan norm_plan(const GroupNormShape& s, bool backward) {
    const int64_t D = s.C / s.groups;
    const int full = s.io == 1 ? 8 : 4;
    NormPlan p;
    p.V = D % full == 0 ? full : (s.io == 1 && D % 2 == 0 ? 2 : 1);
    const int64_t nvec = D / p.V;
    p.LPG = nvec <= 4 ? 4 : nvec <= 8 ? 8 : nvec <= 16 ? 16 : nvec <= 64 ? 32 : nvec <= 128 ? 128 : nvec <= 256 ? 256 : 512;
    p.NV = (p.LPG == 32 && nvec > 32) || (full == 4 && nvec > 512) ? 2 : 1;
    if (p.V < full && p.LPG >= 128) {  // narrow vectors: more of them per lane
        p.LPG = nvec <= 128 ? 32 : nvec <= 256 ? 128 : 256;
        p.NV = nvec <= 128 ? 4 : 2;
    }
    if (nvec > (int64_t)p.LPG * p.NV) p.LPG = 0;
    p.all = p.V == full && nvec == (int64_t)p.LPG * p.NV;
    int64_t most = s.rows, blocks = kSms * 8;
    p.x = s.groups;
    if (p.LPG) {
        blocks = kSms * resident(p.NV * p.V, team_threads(p.LPG), backward);
        if (p.LPG <= 32) {
            p.x = (s.groups + 32 / p.LPG - 1) / (32 / p.LPG);
            most = (s.rows + kTeamWarps - 1) / kTeamWarps;
        }
    }
    int64_t y = blocks / p.x;
    if (y < 1) y = 1;
    p.y = (int)(y < most ? y : most);
    return p;
}

template <typename TIO, int V, int LPG, int NV>
cudaError_t launch_team(const NormPlan& p, const NormArgs& a, bool backward, cudaStream_t s) {
    const dim3 grid((unsigned)p.x, (unsigned)p.y), block(LPG <= 32 ? 32 * kTeamWarps : LPG);
    if constexpr (V * sizeof(TIO) == 16) {
        if (p.all)
            return launch_pdl(backward ? norm_bwd<TIO, V, LPG, NV, true> : norm_fwd<TIO, V, LPG, NV, true>, grid, block, 0, s, a);
    }
    return launch_pdl(backward ? norm_bwd<TIO, V, LPG, NV, false> : norm_fwd<TIO, V, LPG, NV, false>, grid, block, 0, s, a);
}

template <typename TIO, int V>
cudaError_t launch_norm(const NormPlan& p, const NormArgs& a, bool backward, cudaStream_t s) {
    if (p.LPG == 0)
        return launch_pdl(backward ? norm_wide<TIO, V, true> : norm_wide<TIO, V, false>, dim3((unsigned)p.x, (unsigned)p.y),
                          dim3(kWide), 0, s, a);
    if (p.LPG == 4) return launch_team<TIO, V, 4, 1>(p, a, backward, s);
    if (p.LPG == 8) return launch_team<TIO, V, 8, 1>(p, a, backward, s);
    if (p.LPG == 16) return launch_team<TIO, V, 16, 1>(p, a, backward, s);
    if (p.LPG == 32 && p.NV == 1) return launch_team<TIO, V, 32, 1>(p, a, backward, s);
    if (p.LPG == 32 && p.NV == 2) return launch_team<TIO, V, 32, 2>(p, a, backward, s);
    if constexpr (V * sizeof(TIO) == 16) {
        if (p.LPG == 128) return launch_team<TIO, V, 128, 1>(p, a, backward, s);
        if (p.LPG == 256) return launch_team<TIO, V, 256, 1>(p, a, backward, s);
        if constexpr (V == 4)
            if (p.NV == 2) return launch_team<TIO, V, 512, 2>(p, a, backward, s);
        return launch_team<TIO, V, 512, 1>(p, a, backward, s);
    } else {
        if (p.LPG == 32) return launch_team<TIO, V, 32, 4>(p, a, backward, s);
        if (p.LPG == 128) return launch_team<TIO, V, 128, 2>(p, a, backward, s);
        return launch_team<TIO, V, 256, 2>(p, a, backward, s);
    }
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
