// group_norm.cu -- group normalisation, channels last, with an activation or
// an activated gate, forward and backward.
//
//     xh = (x - mean) rstd,  n = xh w + b,   y = act(n)  or  n act(gate)
//     dn = dy act'(n)  or  dy act(gate),     dgate = dy n act'(gate)
//     dw = sum dn xh,  db = sum dn
//     dx = rstd (dn w - mean(dn w) - xh mean(dn w xh))
//
// All bandwidth: each value is touched by a few dozen instructions, so the
// layouts serve wide loads and few passes.
//   Token form (S = 1, group widths up to 8 vectors a lane): a sub-warp of 1
//   to 32 lanes holds one row's group in registers, so x, gate and dy are
//   read once; mean and variance in two passes over the registers.
//   Sample form (S > 1, or wider groups): a pass for the statistics
//   (or the sums of the backward pass), a small join, a second pass that
//   applies them, in the opposite order of blocks so that it starts with what
//   the first pass left in L2.
// Partial results are joined in a fixed order: runs repeat bit for bit.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <string>

#include "../../include/fftconv.h"
#include "internal.h"

namespace fftconv {
namespace {

constexpr int kThreads = 256;

struct Args {
    const void *x, *gate, *w, *b, *dy;
    void *y, *dx, *dgate;
    float *mean, *rstd;          // forward: outputs (may be null in the token form); backward: inputs
    float *part, *sums;          // workspace
    float *dw, *db;
    int64_t N, S, ldx, ldg, ldy;
    int C, G, D;
    int w_f32, act, chunks, parts;
    float eps;
};

template <typename T>
struct Type;
template <>
struct Type<float> {
    static constexpr int Vec = 4;
    static __device__ __forceinline__ float get(float x) { return x; }
    static __device__ __forceinline__ float put(float x) { return x; }
};
template <>
struct Type<__half> {
    static constexpr int Vec = 8;
    static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <>
struct Type<__nv_bfloat16> {
    static constexpr int Vec = 8;
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

// V elements: one 16-byte vector, or one element.
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
    T e[V];
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load(const void* p, int64_t at) {
    Pack<T, V> r;
    if constexpr (V == 1) {
        r.e[0] = reinterpret_cast<const T*>(p)[at];
    } else {
        *reinterpret_cast<uint4*>(&r) = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p) + at);
    }
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void store(void* p, int64_t at, const float (&f)[V]) {
    Pack<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.e[i] = Type<T>::put(f[i]);
    if constexpr (V == 1)
        reinterpret_cast<T*>(p)[at] = r.e[0];
    else
        *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p) + at) = *reinterpret_cast<const uint4*>(&r);
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V>& p, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = Type<T>::get(p.e[i]);
}
// weight or bias of channels c .. c + V (in x's type or fp32)
template <typename T, int V>
__device__ __forceinline__ void load_w(const void* w, int f32, int c, float none, float (&f)[V]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = none;
    } else if (f32) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = reinterpret_cast<const float*>(w)[c + i];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = Type<T>::get(reinterpret_cast<const T*>(w)[c + i]);
    }
}

// exp and the reciprocal of the fast units: both within a few 2^-22 of the
// value for the arguments where the sigmoid is not 0 or 1, below fp32's own
// error of a sum of this kind.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
// act(x) and its slope
__device__ __forceinline__ float activate(float x, int act) {
    if (act == FFTCONV_ACT_NONE) return x;
    const float s = x < -87.f ? 0.f : sigmoid(x);             // (1 + exp would leave __fdividef's range)
    return act == FFTCONV_ACT_SILU ? x * s : s;
}
__device__ __forceinline__ float activate(float x, int act, float& slope) {
    slope = 1.f;
    if (act == FFTCONV_ACT_NONE) return x;
    const float s = x < -87.f ? 0.f : sigmoid(x);
    if (act == FFTCONV_ACT_SIGMOID) {
        slope = s * (1.f - s);
        return s;
    }
    slope = s * fmaf(x, 1.f - s, 1.f);
    return x * s;
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// ------------------------------------------------------------ token form ---

// I vectors of V elements a lane, LANES lanes a (row, group) pair, U pairs in
// flight a sub-warp.
template <typename T, int V, int I, int LANES>
__global__ void __launch_bounds__(kThreads) gn_token_forward(const Args a) {
    constexpr int U = I >= 4 ? 1 : 4 / I;
    const int sub = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    constexpr int kSubs = kThreads / LANES;
    const int nvec = a.D / V;
    const int64_t pairs = a.N * a.G;
    const float inv = 1.f / (float)a.D;
    const int64_t p0 = (int64_t)blockIdx.x * (kSubs * U) + sub;
    Pack<T, V> x[U][I], gt[U][I];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t p = p0 + u * kSubs;
        if (p >= pairs) continue;
        const int64_t r = p / a.G;
        const int c = (int)(p % a.G) * a.D;
#pragma unroll
        for (int i = 0; i < I; ++i)
            if (lane + i * LANES < nvec) {
                const int at = c + (lane + i * LANES) * V;
                x[u][i] = load<T, V>(a.x, r * a.ldx + at);
                if (a.gate) gt[u][i] = load<T, V>(a.gate, r * a.ldg + at);
            }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t p = p0 + u * kSubs;
        const bool in = p < pairs;                            // (all lanes take part in the shuffles)
        const int64_t r = p / a.G;
        const int c = (int)(p % a.G) * a.D;
        float f[I][V], sum = 0.f, sq = 0.f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (in && lane + i * LANES < nvec) {
                unpack<T, V>(x[u][i], f[i]);
#pragma unroll
                for (int j = 0; j < V; ++j) sum += f[i][j];
            }
        }
        const float mean = lanes_sum<LANES>(sum) * inv;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (in && lane + i * LANES < nvec) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    f[i][j] -= mean;
                    sq = fmaf(f[i][j], f[i][j], sq);
                }
            }
        }
        const float rstd = rsqrtf(fmaf(lanes_sum<LANES>(sq), inv, a.eps));
        if (!in) continue;
        if (lane == 0 && a.mean) {
            a.mean[p] = mean;
            a.rstd[p] = rstd;
        }
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (lane + i * LANES >= nvec) continue;
            const int at = c + (lane + i * LANES) * V;
            float w[V], b[V], g[V];
            load_w<T, V>(a.w, a.w_f32, at, 1.f, w);
            load_w<T, V>(a.b, a.w_f32, at, 0.f, b);
            if (a.gate) unpack<T, V>(gt[u][i], g);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float n = fmaf(f[i][j] * rstd, w[j], b[j]);
                f[i][j] = a.gate ? n * activate(g[j], a.act) : activate(n, a.act);
            }
            store<T, V>(a.y, r * a.C + at, f[i]);
        }
    }
}

// Blocks of (groups x rows) sub-warps: a sub-warp keeps its group and walks
// down the rows, so that its channels' dw and db stay in registers.
// blockDim = LANES * subs, subs = gsubs * rsubs; grid (row blocks, group blocks).
template <typename T, int V, int I, int LANES>
__global__ void __launch_bounds__(kThreads) gn_token_backward(const Args a, int gsubs, int rsubs) {
    const int sub = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    const int g = blockIdx.y * gsubs + sub % gsubs, rs = sub / gsubs;
    const bool on = g < a.G && rs < rsubs;
    const int nvec = a.D / V;
    const float inv = 1.f / (float)a.D;
    const int c = g * a.D;
    const int64_t stride = (int64_t)gridDim.x * rsubs;
    const int64_t row0 = (int64_t)blockIdx.x * rsubs;
    float dw[I][V], db[I][V], w[I][V], b[I][V];
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = db[i][j] = w[i][j] = b[i][j] = 0.f;
    if (on)
#pragma unroll
        for (int i = 0; i < I; ++i)
            if (lane + i * LANES < nvec) {
                load_w<T, V>(a.w, a.w_f32, c + (lane + i * LANES) * V, 1.f, w[i]);
                load_w<T, V>(a.b, a.w_f32, c + (lane + i * LANES) * V, 0.f, b[i]);
            }
    for (int64_t base = row0; base < a.N; base += stride) {   // the same trip count for a whole block
        const int64_t r = base + rs;
        const bool in = on && r < a.N;
        float mean = 0.f, rstd = 0.f;
        Pack<T, V> px[I], pd[I], pg[I];
        if (in) {
            mean = a.mean[r * a.G + g];
            rstd = a.rstd[r * a.G + g];
#pragma unroll
            for (int i = 0; i < I; ++i)
                if (lane + i * LANES < nvec) {
                    const int at = c + (lane + i * LANES) * V;
                    px[i] = load<T, V>(a.x, r * a.ldx + at);
                    pd[i] = load<T, V>(a.dy, r * a.ldy + at);
                    if (a.gate) pg[i] = load<T, V>(a.gate, r * a.ldg + at);
                }
        }
        float xh[I][V], dn[I][V], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (!in || lane + i * LANES >= nvec) continue;
            float dy[V], gt[V];
            unpack<T, V>(px[i], xh[i]);
            unpack<T, V>(pd[i], dy);
            if (a.gate) unpack<T, V>(pg[i], gt);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                xh[i][j] = (xh[i][j] - mean) * rstd;
                const float n = fmaf(xh[i][j], w[i][j], b[i][j]);
                float slope;
                if (a.gate) {
                    dn[i][j] = dy[j] * activate(gt[j], a.act, slope);
                    gt[j] = dy[j] * n * slope;
                } else {
                    activate(n, a.act, slope);
                    dn[i][j] = dy[j] * slope;
                }
                dw[i][j] = fmaf(dn[i][j], xh[i][j], dw[i][j]);
                db[i][j] += dn[i][j];
                dn[i][j] *= w[i][j];
                s1 += dn[i][j];
                s2 = fmaf(dn[i][j], xh[i][j], s2);
            }
            if (a.gate) store<T, V>(a.dgate, r * a.C + c + (lane + i * LANES) * V, gt);
        }
        s1 = lanes_sum<LANES>(s1) * inv;
        s2 = lanes_sum<LANES>(s2) * inv;
        if (!in) continue;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (lane + i * LANES >= nvec) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) dn[i][j] = rstd * (dn[i][j] - s1 - xh[i][j] * s2);
            store<T, V>(a.dx, r * a.C + c + (lane + i * LANES) * V, dn[i]);
        }
    }
    if (!on || !a.dw) return;
    float* out = a.part + ((int64_t)blockIdx.x * rsubs + rs) * 2 * a.C + c;
#pragma unroll
    for (int i = 0; i < I; ++i)
        if (lane + i * LANES < nvec)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                out[(lane + i * LANES) * V + j] = dw[i][j];
                out[a.C + (lane + i * LANES) * V + j] = db[i][j];
            }
}

// dw and db: the sum of `parts` rows of (dw[C], db[C]), in a fixed order.
__global__ void __launch_bounds__(1024) gn_sum_parts(const Args a) {
    __shared__ float sh[32][33];
    const int col = blockIdx.x * 32 + threadIdx.x % 32, r0 = threadIdx.x / 32;
    float s = 0.f;
    if (col < 2 * a.C) {
        const float* p = a.part + col;
#pragma unroll 4
        for (int r = r0; r < a.parts; r += 32) s += p[(int64_t)r * 2 * a.C];
    }
    sh[r0][threadIdx.x % 32] = s;
    __syncthreads();
    s = lanes_sum<32>(sh[threadIdx.x % 32][r0]);
    const int c = blockIdx.x * 32 + r0;
    if (threadIdx.x % 32 == 0 && c < 2 * a.C) (c < a.C ? a.dw[c] : a.db[c - a.C]) = s;
}

// ----------------------------------------------------------- sample form ---
//
// A block takes a range of a sample's positions (chunk) and up to 256 vectors
// of its channels: thread = (vector column, row lane).

struct Tile {
    int n, chunk, colv, rl, rows;             // rows: row lanes
    int64_t s0, s1;
    bool on;
};
template <int V>
__device__ __forceinline__ Tile tile_of(const Args& a, int bx) {
    Tile t;
    t.n = bx / a.chunks;
    t.chunk = bx % a.chunks;
    const int cv = a.C / V, width = min(cv - (int)blockIdx.y * kThreads, kThreads);
    t.rows = kThreads / width;
    t.rl = threadIdx.x / width;
    t.colv = blockIdx.y * kThreads + threadIdx.x % width;
    t.on = t.rl < t.rows;
    const int64_t per = (a.S + a.chunks - 1) / a.chunks;
    t.s0 = min((int64_t)t.chunk * per, a.S);
    t.s1 = min(t.s0 + per, a.S);
    return t;
}

// (count, mean, sum of squared deviations) of two sets joined
__device__ __forceinline__ void join(float& n, float& m, float& q, float n2, float m2, float q2) {
    const float t = n + n2;
    if (n2 == 0.f) return;
    const float d = m2 - m, f = n2 / t;
    m = fmaf(d, f, m);
    q += q2 + d * d * n * f;
    n = t;
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) gn_stats(const Args a) {
    __shared__ float sh[3][kThreads];
    const Tile t = tile_of<V>(a, blockIdx.x);
    float n = 0.f, m = 0.f, q = 0.f;
    if (t.on) {
        const int64_t row0 = (int64_t)t.n * a.S;
        constexpr int kAhead = V == 1 ? 8 : 4;
        for (int64_t s = t.s0 + t.rl; s < t.s1; s += (int64_t)t.rows * kAhead) {
            Pack<T, V> p[kAhead];
            float f[kAhead][V], sum = 0.f, sq = 0.f, cnt = 0.f;
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (s + k * t.rows < t.s1) p[k] = load<T, V>(a.x, (row0 + s + k * t.rows) * a.ldx + (int64_t)t.colv * V);
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (s + k * t.rows < t.s1) {
                    unpack<T, V>(p[k], f[k]);
                    cnt += V;
#pragma unroll
                    for (int j = 0; j < V; ++j) sum += f[k][j];
                }
            const float mean = sum / cnt;
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (s + k * t.rows < t.s1)
#pragma unroll
                    for (int j = 0; j < V; ++j) sq = fmaf(f[k][j] - mean, f[k][j] - mean, sq);
            join(n, m, q, cnt, mean, sq);
        }
    }
    sh[0][threadIdx.x] = n;
    sh[1][threadIdx.x] = m;
    sh[2][threadIdx.x] = q;
    __syncthreads();
    // one warp a group: the entries of the group's columns in every row lane
    const int gv = a.D / V, width = min(a.C / V - (int)blockIdx.y * kThreads, kThreads);
    const int v0 = blockIdx.y * kThreads, g0 = v0 / gv, g1 = (v0 + width - 1) / gv;
    const int lane = threadIdx.x % 32;
    for (int g = threadIdx.x / 32; g < a.G; g += kThreads / 32) {
        float gn = 0.f, gm = 0.f, gq = 0.f;
        if (g >= g0 && g <= g1) {
            const int lo = max(g * gv, v0) - v0, hi = min((g + 1) * gv, v0 + width) - v0;
            for (int e = lane; e < (hi - lo) * t.rows; e += 32) {
                const int at = e / (hi - lo) * width + lo + e % (hi - lo);
                join(gn, gm, gq, sh[0][at], sh[1][at], sh[2][at]);
            }
            for (int d = 16; d > 0; d >>= 1) {
                const float n2 = __shfl_down_sync(0xffffffffu, gn, d), m2 = __shfl_down_sync(0xffffffffu, gm, d),
                            q2 = __shfl_down_sync(0xffffffffu, gq, d);
                join(gn, gm, gq, n2, m2, q2);
            }
        }
        if (lane == 0) {
            const int64_t e = ((int64_t)t.n * a.G + g) * a.parts + (int64_t)blockIdx.y * a.chunks + t.chunk;
            reinterpret_cast<float4*>(a.part)[e] = make_float4(gn, gm, gq, 0.f);
        }
    }
}

// One warp a (sample, group): joins its parts.
__global__ void __launch_bounds__(kThreads) gn_join_stats(const Args a) {
    const int64_t p = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    if (p >= a.N * a.G) return;
    const int lane = threadIdx.x % 32;
    float n = 0.f, m = 0.f, q = 0.f;
    for (int e = lane; e < a.parts; e += 32) {
        const float4 v = reinterpret_cast<const float4*>(a.part)[p * a.parts + e];
        join(n, m, q, v.x, v.y, v.z);
    }
    for (int d = 16; d > 0; d >>= 1) {
        const float n2 = __shfl_down_sync(0xffffffffu, n, d), m2 = __shfl_down_sync(0xffffffffu, m, d),
                    q2 = __shfl_down_sync(0xffffffffu, q, d);
        join(n, m, q, n2, m2, q2);
    }
    if (lane == 0) {
        a.mean[p] = m;
        a.rstd[p] = rsqrtf(q / n + a.eps);
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) gn_apply(const Args a) {
    const Tile t = tile_of<V>(a, gridDim.x - 1 - blockIdx.x);
    if (!t.on) return;
    const int c = t.colv * V;
    const int64_t p = (int64_t)t.n * a.G + c / a.D, row0 = (int64_t)t.n * a.S;
    const float mean = a.mean[p], rstd = a.rstd[p];
    float w[V], b[V];
    load_w<T, V>(a.w, a.w_f32, c, 1.f, w);
    load_w<T, V>(a.b, a.w_f32, c, 0.f, b);
    constexpr int kAhead = 4;
    for (int64_t s = t.s0 + t.rl; s < t.s1; s += (int64_t)t.rows * kAhead) {
        Pack<T, V> px[kAhead], pg[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (s + k * t.rows < t.s1) {
                const int64_t r = row0 + s + k * t.rows;
                px[k] = load<T, V>(a.x, r * a.ldx + c);
                if (a.gate) pg[k] = load<T, V>(a.gate, r * a.ldg + c);
            }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (s + k * t.rows < t.s1) {
                float f[V], g[V];
                unpack<T, V>(px[k], f);
                if (a.gate) unpack<T, V>(pg[k], g);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float n = fmaf((f[j] - mean) * rstd, w[j], b[j]);
                    f[j] = a.gate ? n * activate(g[j], a.act) : activate(n, a.act);
                }
                store<T, V>(a.y, (row0 + s + k * t.rows) * a.C + c, f);
            }
    }
}

// dn (and dgate) of one vector
template <typename T, int V>
__device__ __forceinline__ void grad_of(const Args& a, const Pack<T, V>& px, const Pack<T, V>& pd, const Pack<T, V>& pg,
                                        float mean, float rstd, const float (&w)[V], const float (&b)[V],
                                        float (&xh)[V], float (&dn)[V], float (&dg)[V]) {
    float dy[V];
    unpack<T, V>(px, xh);
    unpack<T, V>(pd, dy);
    if (a.gate) unpack<T, V>(pg, dg);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        xh[j] = (xh[j] - mean) * rstd;
        const float n = fmaf(xh[j], w[j], b[j]);
        float slope;
        if (a.gate) {
            dn[j] = dy[j] * activate(dg[j], a.act, slope);
            dg[j] = dy[j] * n * slope;
        } else {
            activate(n, a.act, slope);
            dn[j] = dy[j] * slope;
        }
    }
}

// First backward pass: the sums of dn xh and dn over the chunk's positions,
// by channel: part[(sample, chunk)][2][C].
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) gn_grad_sums(const Args a) {
    __shared__ float sh[2][kThreads][V];
    const Tile t = tile_of<V>(a, blockIdx.x);
    float s1[V], s2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) s1[j] = s2[j] = 0.f;
    const int c = t.colv * V;
    if (t.on) {
        const int64_t p = (int64_t)t.n * a.G + c / a.D, row0 = (int64_t)t.n * a.S;
        const float mean = a.mean[p], rstd = a.rstd[p];
        float w[V], b[V];
        load_w<T, V>(a.w, a.w_f32, c, 1.f, w);
        load_w<T, V>(a.b, a.w_f32, c, 0.f, b);
        constexpr int kAhead = 2;
        for (int64_t s = t.s0 + t.rl; s < t.s1; s += (int64_t)t.rows * kAhead) {
            Pack<T, V> px[kAhead], pd[kAhead], pg[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (s + k * t.rows < t.s1) {
                    const int64_t r = row0 + s + k * t.rows;
                    px[k] = load<T, V>(a.x, r * a.ldx + c);
                    pd[k] = load<T, V>(a.dy, r * a.ldy + c);
                    if (a.gate) pg[k] = load<T, V>(a.gate, r * a.ldg + c);
                }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (s + k * t.rows < t.s1) {
                    float xh[V], dn[V], dg[V];
                    grad_of<T, V>(a, px[k], pd[k], pg[k], mean, rstd, w, b, xh, dn, dg);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        s1[j] = fmaf(dn[j], xh[j], s1[j]);
                        s2[j] += dn[j];
                    }
                }
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        sh[0][threadIdx.x][j] = s1[j];
        sh[1][threadIdx.x][j] = s2[j];
    }
    __syncthreads();
    if (t.on && t.rl == 0) {
        const int width = kThreads / t.rows == 0 ? 1 : min(a.C / V - (int)blockIdx.y * kThreads, kThreads);
        float* out = a.part + (int64_t)blockIdx.x * 2 * a.C + c;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float x = 0.f, y = 0.f;
            for (int r = 0; r < t.rows; ++r) {
                x += sh[0][threadIdx.x + r * width][j];
                y += sh[1][threadIdx.x + r * width][j];
            }
            out[j] = x;
            out[a.C + j] = y;
        }
    }
}

// One warp a (sample, group): mean(dn w) and mean(dn w xh).
template <typename T>
__global__ void __launch_bounds__(kThreads) gn_join_sums(const Args a) {
    const int64_t p = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    if (p >= a.N * a.G) return;
    const int64_t n = p / a.G;
    const int c0 = (int)(p % a.G) * a.D, lane = threadIdx.x % 32;
    float s1 = 0.f, s2 = 0.f;
    for (int c = c0 + lane % a.D; c < c0 + a.D && lane < 32 / min(32, a.D) * a.D; c += 32) {
        // narrow groups: the lanes beyond the first a.D take further chunks
        const int step = a.D >= 32 ? 1 : 32 / a.D;
        float w[1], x = 0.f, y = 0.f;
        load_w<T, 1>(a.w, a.w_f32, c, 1.f, w);
        for (int k = a.D >= 32 ? 0 : lane / a.D; k < a.chunks; k += step) {
            const float* src = a.part + (n * a.chunks + k) * 2 * a.C;
            x += src[c];
            y += src[a.C + c];
        }
        s1 = fmaf(x, w[0], s1);
        s2 = fmaf(y, w[0], s2);
    }
    s1 = lanes_sum<32>(s1);
    s2 = lanes_sum<32>(s2);
    if (lane == 0) {
        const float inv = 1.f / ((float)a.S * (float)a.D);
        a.sums[2 * p] = s2 * inv;
        a.sums[2 * p + 1] = s1 * inv;
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) gn_grad_apply(const Args a) {
    const Tile t = tile_of<V>(a, gridDim.x - 1 - blockIdx.x);
    if (!t.on) return;
    const int c = t.colv * V;
    const int64_t p = (int64_t)t.n * a.G + c / a.D, row0 = (int64_t)t.n * a.S;
    const float mean = a.mean[p], rstd = a.rstd[p], m1 = a.sums[2 * p], m2 = a.sums[2 * p + 1];
    float w[V], b[V];
    load_w<T, V>(a.w, a.w_f32, c, 1.f, w);
    load_w<T, V>(a.b, a.w_f32, c, 0.f, b);
    constexpr int kAhead = 2;
    for (int64_t s = t.s0 + t.rl; s < t.s1; s += (int64_t)t.rows * kAhead) {
        Pack<T, V> px[kAhead], pd[kAhead], pg[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (s + k * t.rows < t.s1) {
                const int64_t r = row0 + s + k * t.rows;
                px[k] = load<T, V>(a.x, r * a.ldx + c);
                pd[k] = load<T, V>(a.dy, r * a.ldy + c);
                if (a.gate) pg[k] = load<T, V>(a.gate, r * a.ldg + c);
            }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (s + k * t.rows < t.s1) {
                const int64_t r = row0 + s + k * t.rows;
                float xh[V], dn[V], dg[V];
                grad_of<T, V>(a, px[k], pd[k], pg[k], mean, rstd, w, b, xh, dn, dg);
                if (a.gate) store<T, V>(a.dgate, r * a.C + c, dg);
#pragma unroll
                for (int j = 0; j < V; ++j) dn[j] = rstd * (dn[j] * w[j] - m1 - xh[j] * m2);
                store<T, V>(a.dx, r * a.C + c, dn);
            }
    }
}

// ------------------------------------------------------------------ host ---

int fail(int status, const std::string& msg) {
    set_last_error(msg.c_str());
    return status;
}

constexpr int64_t kTokenBlocks = 148 * 8;     // row blocks of the token form's backward pass at most

// Samples are cut so that the blocks fill the GPU a few times over, but no
// finer than 16 positions for each row lane.
int64_t chunks_of(int64_t N, int64_t S, int64_t C) {
    int64_t want = (148 * 8 + N - 1) / N;
    const int64_t most = S * C / 16384 > 1 ? S * C / 16384 : 1;
    if (want > most) want = most;
    return want > S ? S : want;
}

// Lanes and vectors a lane of the token form for groups of nvec vectors; 0
// lanes: too wide for it.
void token_shape(int64_t nvec, int& lanes, int& per) {
    lanes = 1;
    while (lanes < 32 && lanes < nvec) lanes *= 2;
    per = 1;
    while (per * lanes < nvec) per *= 2;
    if (per > 8) lanes = 0;
}

template <typename T, int V, int I>
void token_forward(const Args& a, int lanes, cudaStream_t s) {
    constexpr int U = I >= 4 ? 1 : 4 / I;
    const int64_t pairs = a.N * a.G, per = (int64_t)kThreads / lanes * U;
    const unsigned grid = (unsigned)((pairs + per - 1) / per);
    if constexpr (I == 1) {
        switch (lanes) {
            case 1: gn_token_forward<T, V, I, 1><<<grid, kThreads, 0, s>>>(a); return;
            case 2: gn_token_forward<T, V, I, 2><<<grid, kThreads, 0, s>>>(a); return;
            case 4: gn_token_forward<T, V, I, 4><<<grid, kThreads, 0, s>>>(a); return;
            case 8: gn_token_forward<T, V, I, 8><<<grid, kThreads, 0, s>>>(a); return;
            case 16: gn_token_forward<T, V, I, 16><<<grid, kThreads, 0, s>>>(a); return;
            default: break;
        }
    }
    gn_token_forward<T, V, I, 32><<<grid, kThreads, 0, s>>>(a);
}

struct TokenGrid {
    int gsubs, rsubs, threads;
    unsigned gx, gy;
};
TokenGrid token_grid(int64_t N, int64_t G, int lanes) {
    TokenGrid t;
    const int subs = kThreads / lanes;
    t.gsubs = (int)(G < subs ? G : subs);
    t.rsubs = subs / t.gsubs;
    t.threads = (t.gsubs * t.rsubs * lanes + 31) / 32 * 32;
    t.gy = (unsigned)((G + t.gsubs - 1) / t.gsubs);
    int64_t most = kTokenBlocks / t.gy > 1 ? kTokenBlocks / t.gy : 1;
    const int64_t rows = (N + t.rsubs - 1) / t.rsubs;
    t.gx = (unsigned)(rows < most ? rows : most);
    return t;
}

template <typename T, int V, int I>
void token_backward(const Args& a, int lanes, const TokenGrid& t, cudaStream_t s) {
    const dim3 grid(t.gx, t.gy);
    if constexpr (I == 1) {
        switch (lanes) {
            case 1: gn_token_backward<T, V, I, 1><<<grid, t.threads, 0, s>>>(a, t.gsubs, t.rsubs); return;
            case 2: gn_token_backward<T, V, I, 2><<<grid, t.threads, 0, s>>>(a, t.gsubs, t.rsubs); return;
            case 4: gn_token_backward<T, V, I, 4><<<grid, t.threads, 0, s>>>(a, t.gsubs, t.rsubs); return;
            case 8: gn_token_backward<T, V, I, 8><<<grid, t.threads, 0, s>>>(a, t.gsubs, t.rsubs); return;
            case 16: gn_token_backward<T, V, I, 16><<<grid, t.threads, 0, s>>>(a, t.gsubs, t.rsubs); return;
            default: break;
        }
    }
    gn_token_backward<T, V, I, 32><<<grid, t.threads, 0, s>>>(a, t.gsubs, t.rsubs);
}

template <typename T, int V>
void forward(Args a, bool token, int lanes, int per, cudaStream_t s) {
    if (token) {
        switch (per) {
            case 1: return token_forward<T, V, 1>(a, lanes, s);
            case 2: return token_forward<T, V, 2>(a, lanes, s);
            case 4: return token_forward<T, V, 4>(a, lanes, s);
            default: return token_forward<T, V, 8>(a, lanes, s);
        }
    }
    const unsigned cols = (unsigned)((a.C / V + kThreads - 1) / kThreads);
    const dim3 grid((unsigned)(a.N * a.chunks), cols);
    a.parts = (int)cols * a.chunks;
    gn_stats<T, V><<<grid, kThreads, 0, s>>>(a);
    gn_join_stats<<<(unsigned)((a.N * a.G + 7) / 8), kThreads, 0, s>>>(a);
    gn_apply<T, V><<<grid, kThreads, 0, s>>>(a);
}

template <typename T, int V>
void backward(Args a, bool token, int lanes, int per, cudaStream_t s) {
    if (token) {
        const TokenGrid t = token_grid(a.N, a.G, lanes);
        a.parts = (int)t.gx * t.rsubs;
        switch (per) {
            case 1: token_backward<T, V, 1>(a, lanes, t, s); break;
            case 2: token_backward<T, V, 2>(a, lanes, t, s); break;
            case 4: token_backward<T, V, 4>(a, lanes, t, s); break;
            default: token_backward<T, V, 8>(a, lanes, t, s); break;
        }
    } else {
        const unsigned cols = (unsigned)((a.C / V + kThreads - 1) / kThreads);
        const dim3 grid((unsigned)(a.N * a.chunks), cols);
        a.parts = (int)(a.N * a.chunks);
        gn_grad_sums<T, V><<<grid, kThreads, 0, s>>>(a);
        gn_join_sums<T><<<(unsigned)((a.N * a.G + 7) / 8), kThreads, 0, s>>>(a);
        gn_grad_apply<T, V><<<grid, kThreads, 0, s>>>(a);
    }
    if (a.dw) gn_sum_parts<<<(unsigned)((2 * a.C + 31) / 32), 1024, 0, s>>>(a);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int64_t pad256(int64_t b) { return (b + 255) / 256 * 256; }

int vec_of(int dtype) { return dtype == FFTCONV_F32 ? 4 : 8; }

// The token form serves both vector widths by the same rule; its width
// depends on alignment, so the workspace is sized for either form.
size_t workspace_bytes(int64_t N, int64_t S, int64_t C, int64_t G, bool bwd) {
    if (N == 0 || S == 0 || C == 0) return 0;
    const int64_t chunks = chunks_of(N, S, C);
    // (groups of up to 256 channels of one position take the token form whatever their alignment)
    if (!bwd && S == 1 && C / G <= 256) return 0;
    if (!bwd) {
        // parts of the statistics, and mean and rstd when the caller keeps none
        return (size_t)(pad256(N * G * chunks * ((C + kThreads - 1) / kThreads) * 16) + 2 * pad256(N * G * 4));
    }
    int64_t parts = N * chunks;
    if (S == 1 && parts > kTokenBlocks * kThreads) parts = N;
    const int64_t token = S == 1 ? (N < kTokenBlocks * kThreads ? N + kThreads : kTokenBlocks * kThreads) : 0;
    if (token > parts) parts = token;
    return (size_t)(pad256(parts * 2 * C * 4) + pad256(N * G * 8));
}

int check(int64_t N, int64_t S, int64_t C, int64_t G, int dtype, int wdtype, int act, bool affine) {
    if (N < 0 || S < 0 || C <= 0 || G <= 0) return fail(FFTCONV_ERR_INVALID_ARG, "N, S, C or G out of range");
    if (C % G) return fail(FFTCONV_ERR_INVALID_ARG, "G must divide C");
    if (dtype != FFTCONV_F32 && dtype != FFTCONV_F16 && dtype != FFTCONV_BF16)
        return fail(FFTCONV_ERR_INVALID_ARG, "unknown dtype");
    if (affine && wdtype != dtype && wdtype != FFTCONV_F32)
        return fail(FFTCONV_ERR_INVALID_ARG, "weight and bias must have x's type or fp32");
    if (act < FFTCONV_ACT_NONE || act > FFTCONV_ACT_SIGMOID) return fail(FFTCONV_ERR_INVALID_ARG, "unknown activation");
    if (C >= (int64_t(1) << 24) || (double)N * (double)G >= 2147483647.0 ||
        (double)N * (double)chunks_of(N ? N : 1, S ? S : 1, C) >= 2147483647.0)
        return fail(FFTCONV_ERR_UNSUPPORTED, "too many channels, samples or groups");
    return FFTCONV_OK;
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

template <typename F>
void dispatch(int dtype, bool vec, F&& f) {
    if (dtype == FFTCONV_F32)
        vec ? f((float*)nullptr, std::integral_constant<int, 4>{}) : f((float*)nullptr, std::integral_constant<int, 1>{});
    else if (dtype == FFTCONV_F16)
        vec ? f((__half*)nullptr, std::integral_constant<int, 8>{}) : f((__half*)nullptr, std::integral_constant<int, 1>{});
    else
        vec ? f((__nv_bfloat16*)nullptr, std::integral_constant<int, 8>{})
            : f((__nv_bfloat16*)nullptr, std::integral_constant<int, 1>{});
}

}  // namespace
}  // namespace fftconv

using namespace fftconv;

extern "C" {

size_t fftconv_group_norm_workspace_bytes(int64_t N, int64_t S, int64_t C, int64_t G, int backward) {
    if (N < 0 || S < 0 || C <= 0 || G <= 0 || C % G) return 0;
    return workspace_bytes(N, S, C, G, backward != 0);
}

int fftconv_group_norm(const void* x, const void* gate, const void* weight, const void* bias, void* y, float* mean,
                       float* rstd, int64_t N, int64_t S, int64_t C, int64_t G, int64_t ld_x, int64_t ld_gate,
                       fftconv_dtype_t dtype, fftconv_dtype_t weight_dtype, fftconv_activation_t act, float eps,
                       void* workspace, size_t workspace_size, fftconv_stream_t stream) {
    set_last_error("");
    if (int e = check(N, S, C, G, dtype, weight_dtype, act, weight != nullptr)) return e;
    if (!weight != !bias) return fail(FFTCONV_ERR_INVALID_ARG, "weight and bias: both or neither");
    if (!mean != !rstd) return fail(FFTCONV_ERR_INVALID_ARG, "mean and rstd: both or neither");
    if (N == 0 || S == 0) return FFTCONV_OK;
    if (!x || !y) return fail(FFTCONV_ERR_INVALID_ARG, "x and y must be non-NULL");
    if (!aligned16(x) || !aligned16(gate) || !aligned16(y) || !aligned16(weight) || !aligned16(bias))
        return fail(FFTCONV_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
    const int64_t rows = N * S, es = dtype == FFTCONV_F32 ? 4 : 2;
    if ((rows > 1 && ld_x < C) || (gate && rows > 1 && ld_gate < C))
        return fail(FFTCONV_ERR_INVALID_ARG, "a row stride is smaller than a row");
    const int64_t bytes = rows * C * es;
    if (overlap(y, bytes, x, ((rows - 1) * ld_x + C) * es) || overlap(y, bytes, gate, ((rows - 1) * ld_gate + C) * es))
        return fail(FFTCONV_ERR_INVALID_ARG, "y overlaps an input");
    const size_t need = workspace_bytes(N, S, C, G, false);
    if (need && (!workspace || workspace_size < need))
        return fail(FFTCONV_ERR_INVALID_ARG, "workspace of " + std::to_string(workspace_size) + " bytes, " +
                                                 std::to_string(need) + " needed");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(FFTCONV_ERR_ALIGNMENT, "workspace not 256-byte aligned");
    Args a{};
    a.x = x; a.gate = gate; a.w = weight; a.b = bias; a.y = y;
    a.N = N; a.S = S; a.C = (int)C; a.G = (int)G; a.D = (int)(C / G);
    a.ldx = ld_x; a.ldg = ld_gate;
    a.w_f32 = weight_dtype == FFTCONV_F32;
    a.act = act;
    a.eps = eps;
    a.chunks = (int)chunks_of(N, S, C);
    const int V = vec_of(dtype);
    const bool vec = a.D % V == 0 && (rows == 1 || ld_x % V == 0) && (!gate || rows == 1 || ld_gate % V == 0);
    int lanes = 0, per = 0;
    token_shape(a.D / (vec ? V : 1), lanes, per);
    const bool token = S == 1 && lanes > 0;
    a.mean = mean;
    a.rstd = rstd;
    if (!token) {
        const int64_t parts = pad256(N * G * (int64_t)a.chunks * ((C + kThreads - 1) / kThreads) * 16);
        a.part = (float*)workspace;
        if (!mean) {
            a.mean = (float*)((uint8_t*)workspace + parts);
            a.rstd = (float*)((uint8_t*)workspace + parts + pad256(N * G * 4));
        }
    }
    dispatch(dtype, vec, [&](auto* t, auto v) {
        using T = std::remove_pointer_t<decltype(t)>;
        forward<T, decltype(v)::value>(a, token, lanes, per, (cudaStream_t)stream);
    });
    const cudaError_t e = cudaPeekAtLastError();
    return e == cudaSuccess ? FFTCONV_OK
                            : fail(FFTCONV_ERR_CUDA, std::string("group norm launch: ") + cudaGetErrorString(e));
}

int fftconv_group_norm_backward(const void* x, const void* gate, const void* weight, const void* bias, const void* dy,
                                const float* mean, const float* rstd, void* dx, void* dgate, float* dweight,
                                float* dbias, int64_t N, int64_t S, int64_t C, int64_t G, int64_t ld_x,
                                int64_t ld_gate, int64_t ld_dy, fftconv_dtype_t dtype, fftconv_dtype_t weight_dtype,
                                fftconv_activation_t act, void* workspace, size_t workspace_size,
                                fftconv_stream_t stream) {
    set_last_error("");
    if (int e = check(N, S, C, G, dtype, weight_dtype, act, weight != nullptr)) return e;
    if (!weight != !bias) return fail(FFTCONV_ERR_INVALID_ARG, "weight and bias: both or neither");
    if (!dweight != !dbias) return fail(FFTCONV_ERR_INVALID_ARG, "dweight and dbias: both or neither");
    if (dweight && !weight) return fail(FFTCONV_ERR_INVALID_ARG, "dweight without weight");
    if (!gate != !dgate) return fail(FFTCONV_ERR_INVALID_ARG, "gate and dgate: both or neither");
    cudaStream_t s = (cudaStream_t)stream;
    if (N == 0 || S == 0) {
        cudaError_t e = cudaSuccess;
        if (dweight) e = cudaMemsetAsync(dweight, 0, (size_t)C * 4, s);
        if (dweight && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, (size_t)C * 4, s);
        return e == cudaSuccess ? FFTCONV_OK : fail(FFTCONV_ERR_CUDA, cudaGetErrorString(e));
    }
    if (!x || !dy || !mean || !rstd || !dx)
        return fail(FFTCONV_ERR_INVALID_ARG, "x, dy, mean, rstd and dx must be non-NULL");
    if (!aligned16(x) || !aligned16(gate) || !aligned16(dy) || !aligned16(dx) || !aligned16(dgate) ||
        !aligned16(weight) || !aligned16(bias))
        return fail(FFTCONV_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
    const int64_t rows = N * S, es = dtype == FFTCONV_F32 ? 4 : 2;
    if (rows > 1 && (ld_x < C || ld_dy < C || (gate && ld_gate < C)))
        return fail(FFTCONV_ERR_INVALID_ARG, "a row stride is smaller than a row");
    const int64_t bytes = rows * C * es;
    const void* in[3] = {x, dy, gate};
    const int64_t ld[3] = {ld_x, ld_dy, ld_gate};
    for (int i = 0; i < 3; ++i)
        if (overlap(dx, bytes, in[i], ((rows - 1) * ld[i] + C) * es) ||
            overlap(dgate, bytes, in[i], ((rows - 1) * ld[i] + C) * es))
            return fail(FFTCONV_ERR_INVALID_ARG, "a gradient overlaps an input");
    if (overlap(dx, bytes, dgate, bytes)) return fail(FFTCONV_ERR_INVALID_ARG, "dx overlaps dgate");
    const size_t need = workspace_bytes(N, S, C, G, true);
    if (need && (!workspace || workspace_size < need))
        return fail(FFTCONV_ERR_INVALID_ARG, "workspace of " + std::to_string(workspace_size) + " bytes, " +
                                                 std::to_string(need) + " needed");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(FFTCONV_ERR_ALIGNMENT, "workspace not 256-byte aligned");
    Args a{};
    a.x = x; a.gate = gate; a.w = weight; a.b = bias; a.dy = dy;
    a.dx = dx; a.dgate = dgate; a.dw = dweight; a.db = dbias;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.N = N; a.S = S; a.C = (int)C; a.G = (int)G; a.D = (int)(C / G);
    a.ldx = ld_x; a.ldg = ld_gate; a.ldy = ld_dy;
    a.w_f32 = weight_dtype == FFTCONV_F32;
    a.act = act;
    a.chunks = (int)chunks_of(N, S, C);
    const int V = vec_of(dtype);
    const bool vec = a.D % V == 0 && (rows == 1 || (ld_x % V == 0 && ld_dy % V == 0 && (!gate || ld_gate % V == 0)));
    int lanes = 0, per = 0;
    token_shape(a.D / (vec ? V : 1), lanes, per);
    const bool token = S == 1 && lanes > 0;
    a.sums = (float*)workspace;
    a.part = (float*)((uint8_t*)workspace + pad256(N * G * 8));
    dispatch(dtype, vec, [&](auto* t, auto v) {
        using T = std::remove_pointer_t<decltype(t)>;
        backward<T, decltype(v)::value>(a, token, lanes, per, s);
    });
    const cudaError_t e = cudaPeekAtLastError();
    return e == cudaSuccess ? FFTCONV_OK
                            : fail(FFTCONV_ERR_CUDA, std::string("group norm backward launch: ") + cudaGetErrorString(e));
}

}  // extern "C"
