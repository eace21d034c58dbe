// group_norm.cu -- group normalisation, channels last, with an activation or
// an activated gate, forward and backward.
//
//     xh = (x - mean) rstd,  n = xh w + b,   y = act(n)  or  n act(gate)
//     dn = dy act'(n)  or  dy act(gate),     dgate = dy n act'(gate)
//     dw = sum dn xh,  db = sum dn
//     dx = rstd (dn w - mean(dn w) - xh mean(dn w xh))
//
// All bandwidth: each value is touched by a few dozen instructions, so the
// layouts serve wide loads, few passes and few instructions.
//   Token form (S = 1, groups of up to 512 channels): a sub-warp of 1 to 32
//   lanes keeps its group, with the group's weights (and sums of dw and db) in
//   registers, and walks down the rows; x, gate and dy are read once, mean and
//   variance take two passes over the registers.
//   Sample form (S > 1, or wider groups): a pass for the statistics (or the
//   sums of the backward pass), a small join, a second pass that applies them,
//   in the opposite order so that it starts with what the first pass left in
//   L2.  A thread keeps its channels, so groups need not be whole vectors.
// Arithmetic is packed, two fp32 values an instruction: with one at a time the
// statistics took 15 instructions a value and the issue slots were the bound
// (73 % of them used; 16 x 4095 x 760 fp16: 32.5 us, packed 28.6).  Results
// are written, and data read for the last time is read, with streaming
// accesses, which leave L2 to what the next pass reads (backward pass of
// 32768 x 2048 bf16 with a gate: 147 -> 137 us).
// Partial results are joined in a fixed order: runs repeat bit for bit.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <string>
#include <type_traits>

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
    int add;                     // dw and db are added to (samples before these)
    int keep;                    // forward: mean and rstd are the caller's
    float eps;
};

template <typename T>
__device__ __forceinline__ float get(T x) {
    if constexpr (std::is_same_v<T, float>) return x;
    else if constexpr (std::is_same_v<T, __half>) return __half2float(x);
    else return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T put(float x) {
    if constexpr (std::is_same_v<T, float>) return x;
    else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(x);
    else return __float2bfloat16_rn(x);
}

// V elements: one 16-byte vector, as the words it is loaded in, or one element.
template <typename T, int V>
struct Pack {
    uint32_t w[V == 1 ? 1 : 4];
};
// (LAST: no later pass reads it, so it need not stay in L2)
template <typename T, int V, bool LAST = false>
__device__ __forceinline__ Pack<T, V> load(const void* p, int64_t at) {
    Pack<T, V> r;
    if constexpr (V > 1) {
        const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p) + at);
        const uint4 v = LAST ? __ldcs(src) : *src;
        r.w[0] = v.x;
        r.w[1] = v.y;
        r.w[2] = v.z;
        r.w[3] = v.w;
    } else if constexpr (sizeof(T) == 4) {
        r.w[0] = reinterpret_cast<const uint32_t*>(p)[at];
    } else {
        r.w[0] = reinterpret_cast<const uint16_t*>(p)[at];
    }
    return r;
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> pack_of(const uint4& v) {
    Pack<T, V> p;
    p.w[0] = v.x;
    if constexpr (V > 1) {
        p.w[1] = v.y;
        p.w[2] = v.z;
        p.w[3] = v.w;
    }
    return p;
}
template <typename T>
__device__ __forceinline__ float2 two_of(uint32_t w) {
    if constexpr (std::is_same_v<T, __half>) {
        __half2 h;
        *reinterpret_cast<uint32_t*>(&h) = w;
        return __half22float2(h);
    } else {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V>& p, float (&f)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = __uint_as_float(p.w[i]);
    } else if constexpr (V == 1) {
        f[0] = two_of<T>(p.w[0]).x;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = two_of<T>(p.w[i]);
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
}
template <typename T, int V>
__device__ __forceinline__ void store(void* p, int64_t at, const float (&f)[V]) {
    if constexpr (V == 1) {
        reinterpret_cast<T*>(p)[at] = put<T>(f[0]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4)
                w[i] = __float_as_uint(f[i]);
            else if constexpr (std::is_same_v<T, __half>)
                asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
            else
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
        }
        __stcs(reinterpret_cast<uint4*>(reinterpret_cast<T*>(p) + at), make_uint4(w[0], w[1], w[2], w[3]));
    }
}
// weight or bias of channels c .. c + V (in x's type or fp32)
template <typename T, int V>
__device__ __forceinline__ void load_w(const void* w, int f32, int c, float none, float (&f)[V]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = none;
    } else if (f32) {
        const float* p = reinterpret_cast<const float*>(w) + c;
        if constexpr (V == 1) {
            f[0] = p[0];
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(p + i);
                f[i] = v.x;
                f[i + 1] = v.y;
                f[i + 2] = v.z;
                f[i + 3] = v.w;
            }
        }
    } else {
        const Pack<T, V> v = load<T, V>(w, c);
        unpack<T, V>(v, f);
    }
}

// fp32 arithmetic on V elements, two an instruction.  A second operand of one
// element stands for all.
__device__ __forceinline__ uint64_t two(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void split(uint64_t r, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
}
template <int V, int N>
__device__ __forceinline__ uint64_t two(const float (&f)[N], int j) {
    static_assert(N == V || N == 1);
    return N == 1 ? two(f[0], f[0]) : two(f[j], f[j + (N > 1)]);
}
// r = a b + c
template <int V, int NB, int NC>
__device__ __forceinline__ void fma_v(float (&r)[V], const float (&a)[V], const float (&b)[NB], const float (&c)[NC]) {
    if constexpr (V == 1) {
        r[0] = fmaf(a[0], b[0], c[0]);
    } else {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            uint64_t d;
            asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(two<V>(a, j)), "l"(two<V>(b, j)), "l"(two<V>(c, j)));
            split(d, r[j], r[j + 1]);
        }
    }
}
template <int V, int NB>
__device__ __forceinline__ void mul_v(float (&r)[V], const float (&a)[V], const float (&b)[NB]) {
    if constexpr (V == 1) {
        r[0] = a[0] * b[0];
    } else {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            uint64_t d;
            asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(two<V>(a, j)), "l"(two<V>(b, j)));
            split(d, r[j], r[j + 1]);
        }
    }
}
template <int V, int NB>
__device__ __forceinline__ void add_v(float (&r)[V], const float (&a)[V], const float (&b)[NB]) {
    if constexpr (V == 1) {
        r[0] = a[0] + b[0];
    } else {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            uint64_t d;
            asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(two<V>(a, j)), "l"(two<V>(b, j)));
            split(d, r[j], r[j + 1]);
        }
    }
}
// the sum of V elements
template <int V>
__device__ __forceinline__ float sum_v(const float (&f)[V]) {
    if constexpr (V == 1) {
        return f[0];
    } else {
        float h[V / 2], k[V / 2];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            h[j] = f[j];
            k[j] = f[j + V / 2];
        }
        add_v<V / 2>(h, h, k);
        return sum_v<V / 2>(h);
    }
}

// s = 1 / (1 + exp(-f)) with the fast units' exp2 and reciprocal: both within
// a few 2^-22 of the value for the arguments where the sigmoid is not 0 or 1,
// below fp32's own error of a sum of this kind.  (An infinite exp gives 0.)
template <int V>
__device__ __forceinline__ void sigmoid(const float (&f)[V], float (&s)[V]) {
    const float scale[1] = {-1.4426950408889634f}, one[1] = {1.f};
    mul_v<V>(s, f, scale);
#pragma unroll
    for (int j = 0; j < V; ++j) asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(s[j]));
    add_v<V>(s, s, one);
#pragma unroll
    for (int j = 0; j < V; ++j) asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(s[j]));
}

// f <- act(f); slope (if wanted): act'.  One uniform branch a vector.
template <int V, bool SLOPE>
__device__ __forceinline__ void activate(float (&f)[V], float (&slope)[V], int act) {
    const float one[1] = {1.f}, minus[1] = {-1.f};
    if (act == FFTCONV_ACT_NONE) {
        if (SLOPE)
#pragma unroll
            for (int j = 0; j < V; ++j) slope[j] = 1.f;
    } else if (act == FFTCONV_ACT_SILU) {
        float s[V];
        sigmoid<V>(f, s);
        mul_v<V>(f, f, s);
        if (SLOPE) {                                          // s + f s (1 - s)
            fma_v<V>(slope, s, minus, one);
            fma_v<V>(slope, f, slope, s);
        }
    } else {
        float s[V];
        sigmoid<V>(f, s);
        if (SLOPE) {
            fma_v<V>(slope, s, minus, one);
            mul_v<V>(slope, slope, s);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = s[j];
    }
}
// y of n (in place): act(n), or n act(gate)
template <int V, bool GATED>
__device__ __forceinline__ void finish(float (&n)[V], float (&gate)[V], int act) {
    float none[V];
    if constexpr (GATED) {
        activate<V, false>(gate, none, act);
        mul_v<V>(n, n, gate);
    } else {
        activate<V, false>(n, none, act);
    }
}
// dn of dy (in place), and dgate of the gate (in place)
template <int V, bool GATED>
__device__ __forceinline__ void start(float (&n)[V], float (&dy)[V], float (&gate)[V], int act) {
    float slope[V];
    if constexpr (GATED) {
        activate<V, true>(gate, slope, act);
        mul_v<V>(n, n, slope);
        mul_v<V>(n, n, dy);
        mul_v<V>(dy, dy, gate);
#pragma unroll
        for (int j = 0; j < V; ++j) gate[j] = n[j];
    } else {
        activate<V, true>(n, slope, act);
        mul_v<V>(dy, dy, slope);
    }
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// ------------------------------------------------------------ token form ---
//
// I vectors of V elements a lane, LANES lanes a group.  Blocks of
// gsubs x rsubs sub-warps (groups x rows), grid (row blocks, group blocks); U
// rows of a sub-warp are in flight together.

template <typename T, int V, int I, int LANES, bool GATED>
__global__ void __launch_bounds__(kThreads, I == 1 ? 3 : 2) gn_token_forward(const Args a, int gsubs, int rsubs) {
    constexpr int U = I == 1 ? 2 : 1;
    constexpr bool kKeep = I * V <= 16;                       // weights stay in registers
    const int sub = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    const int g = blockIdx.y * gsubs + sub % gsubs, rs = sub / gsubs;
    const bool on = g < a.G && rs < rsubs;
    const int nvec = a.D / V, c = g * a.D + lane * V;
    const float inv = 1.f / (float)a.D;
    float w[kKeep ? I : 1][V], b[kKeep ? I : 1][V];
    if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < I; ++i)
            if (on && lane + i * LANES < nvec) {
                load_w<T, V>(a.w, a.w_f32, c + i * LANES * V, 1.f, w[i]);
                load_w<T, V>(a.b, a.w_f32, c + i * LANES * V, 0.f, b[i]);
            }
    }
    Pack<T, V> x[U][I], gt[U][I], nx[U][I], ng[U][I];
    auto fetch = [&](int64_t base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = base + u * rsubs + rs;
#pragma unroll
            for (int i = 0; i < I; ++i)
                if (on && r < a.N && lane + i * LANES < nvec) {
                    nx[u][i] = load<T, V>(a.x, r * a.ldx + c + i * LANES * V);
                    if constexpr (GATED) ng[u][i] = load<T, V>(a.gate, r * a.ldg + c + i * LANES * V);
                }
        }
    };
    const int64_t stride = (int64_t)gridDim.x * rsubs * U;
    fetch((int64_t)blockIdx.x * rsubs * U);
    // (the same trip count for a whole block: all lanes take part in the sums)
    for (int64_t base = (int64_t)blockIdx.x * rsubs * U; base < a.N; base += stride) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < I; ++i) {
                x[u][i] = nx[u][i];
                gt[u][i] = ng[u][i];
            }
        fetch(base + stride);                                 // the next rows' loads are out during this one's work
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = base + u * rsubs + rs;
            const bool in = on && r < a.N;
            float f[I][V], sum = 0.f, sq = 0.f;
#pragma unroll
            for (int i = 0; i < I; ++i)
                if (in && lane + i * LANES < nvec) {
                    unpack<T, V>(x[u][i], f[i]);
                    sum += sum_v<V>(f[i]);
                }
            const float mean = lanes_sum<LANES>(sum) * inv, minus_mean[1] = {-mean};
#pragma unroll
            for (int i = 0; i < I; ++i)
                if (in && lane + i * LANES < nvec) {
                    float f2[V];
                    add_v<V>(f[i], f[i], minus_mean);
                    mul_v<V>(f2, f[i], f[i]);
                    sq += sum_v<V>(f2);
                }
            const float rstd = rsqrtf(fmaf(lanes_sum<LANES>(sq), inv, a.eps)), scale[1] = {rstd};
            if (!in) continue;
            if (lane == 0 && a.mean) {
                a.mean[r * a.G + g] = mean;
                a.rstd[r * a.G + g] = rstd;
            }
#pragma unroll
            for (int i = 0; i < I; ++i) {
                if (lane + i * LANES >= nvec) continue;
                float gate[V];
                if constexpr (GATED) unpack<T, V>(gt[u][i], gate);
                mul_v<V>(f[i], f[i], scale);
                if constexpr (kKeep) {
                    fma_v<V>(f[i], f[i], w[i], b[i]);
                } else {
                    float wi[V], bi[V];
                    load_w<T, V>(a.w, a.w_f32, c + i * LANES * V, 1.f, wi);
                    load_w<T, V>(a.b, a.w_f32, c + i * LANES * V, 0.f, bi);
                    fma_v<V>(f[i], f[i], wi, bi);
                }
                finish<V, GATED>(f[i], gate, a.act);
                store<T, V>(a.y, r * a.C + c + i * LANES * V, f[i]);
            }
        }
    }
}

template <typename T, int V, int I, int LANES, bool GATED>
__global__ void __launch_bounds__(kThreads, I* V <= 8 ? 3 : 2) gn_token_backward(const Args a, int gsubs, int rsubs) {
    const int sub = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    const int g = blockIdx.y * gsubs + sub % gsubs, rs = sub / gsubs;
    const bool on = g < a.G && rs < rsubs;
    const int nvec = a.D / V, c = g * a.D + lane * V;
    const float inv = 1.f / (float)a.D;
    // a lane's own weights: in shared memory where they would crowd out the
    // registers of a third block (vectors of 8)
    constexpr bool kShared = I * V >= 8;
    __shared__ float4 shw[kShared ? I * V / 4 : 1][kThreads], shb[kShared ? I * V / 4 : 1][kThreads];
    float dw[I][V], db[I][V], w[kShared ? 1 : I][V], b[kShared ? 1 : I][V];
#pragma unroll
    for (int i = 0; i < I; ++i) {
        float wi[V], bi[V];
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = db[i][j] = wi[j] = bi[j] = 0.f;
        if (on && lane + i * LANES < nvec) {
            load_w<T, V>(a.w, a.w_f32, c + i * LANES * V, 1.f, wi);
            load_w<T, V>(a.b, a.w_f32, c + i * LANES * V, 0.f, bi);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if constexpr (kShared) {
                reinterpret_cast<float*>(&shw[(i * V + j) / 4][threadIdx.x])[(i * V + j) % 4] = wi[j];
                reinterpret_cast<float*>(&shb[(i * V + j) / 4][threadIdx.x])[(i * V + j) % 4] = bi[j];
            } else {
                w[i][j] = wi[j];
                b[i][j] = bi[j];
            }
        }
    }
    auto own = [&](const float4 (*sh)[kThreads], int i, float (&f)[V]) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if constexpr (V % 4 == 0) {
                if (j % 4 == 0) {
                    const float4 v = sh[(i * V + j) / 4][threadIdx.x];
                    f[j] = v.x;
                    f[j + 1] = v.y;
                    f[j + 2] = v.z;
                    f[j + 3] = v.w;
                }
            } else {
                f[j] = reinterpret_cast<const float*>(&sh[(i * V + j) / 4][threadIdx.x])[(i * V + j) % 4];
            }
        }
    };
    // Rows come D ahead: by asynchronous copies into a lane's own slots in
    // shared memory where those fit beside the weights, else in registers.
    // (Loads in flight were the bound, 5.6 of 11 cycles between a warp's
    // instructions: 32768 x 2048 bf16 with a gate, one row ahead in registers
    // 141 us, two in shared memory 126, of 104 for the bytes.)
    constexpr bool kRing = V > 1 && I == 1;
    constexpr int D = kRing ? 2 : 1, kVecs = (GATED ? 3 : 2) * I;
    __shared__ uint4 slots[kRing ? D * kVecs : 1][kRing ? kThreads : 1];
    float means[D], rstds[D];
    Pack<T, V> px[I], pd[I], pg[I];
    auto bring = [&](Pack<T, V>& reg, int slot, const void* from, int64_t at) {
        if constexpr (kRing)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             (uint32_t)__cvta_generic_to_shared(&slots[slot][threadIdx.x])),
                         "l"(reinterpret_cast<const T*>(from) + at)
                         : "memory");
        else
            reg = load<T, V, true>(from, at);
    };
    auto fetch = [&](int d, int64_t r) {
        if (on && r < a.N) {
            means[d] = a.mean[r * a.G + g];
            rstds[d] = a.rstd[r * a.G + g];
#pragma unroll
            for (int i = 0; i < I; ++i)
                if (lane + i * LANES < nvec) {
                    const int at = c + i * LANES * V, slot = d * kVecs + i;
                    bring(px[i], slot, a.x, r * a.ldx + at);
                    bring(pd[i], slot + I, a.dy, r * a.ldy + at);
                    if constexpr (GATED) bring(pg[i], slot + 2 * I, a.gate, r * a.ldg + at);
                }
        }
        if constexpr (kRing) asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int64_t stride = (int64_t)gridDim.x * rsubs;
    auto row = [&](int d, int64_t r) {
        const bool in = on && r < a.N;
        if constexpr (kRing) asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
        const float minus_mean[1] = {-means[d]}, scale[1] = {rstds[d]};
        float xh[I][V], dn[I][V], gt[I][V], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < I; ++i)
            if (in && lane + i * LANES < nvec) {
                if constexpr (kRing) {
                    const int slot = d * kVecs + i;
                    px[i] = pack_of<T, V>(slots[slot][threadIdx.x]);
                    pd[i] = pack_of<T, V>(slots[slot + I][threadIdx.x]);
                    if constexpr (GATED) pg[i] = pack_of<T, V>(slots[slot + 2 * I][threadIdx.x]);
                }
                unpack<T, V>(px[i], xh[i]);
                unpack<T, V>(pd[i], dn[i]);
                if constexpr (GATED) unpack<T, V>(pg[i], gt[i]);
                add_v<V>(xh[i], xh[i], minus_mean);
                mul_v<V>(xh[i], xh[i], scale);
            }
        if constexpr (!kRing) fetch(d, r + D * stride);       // the next row's loads are out during this one's work
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (!in || lane + i * LANES >= nvec) continue;
            float n[V], wi[V], bi[V];
            if constexpr (kShared) {
                own(shw, i, wi);
                own(shb, i, bi);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    wi[j] = w[i][j];
                    bi[j] = b[i][j];
                }
            }
            fma_v<V>(n, xh[i], wi, bi);
            start<V, GATED>(n, dn[i], gt[i], a.act);
            fma_v<V>(dw[i], dn[i], xh[i], dw[i]);
            add_v<V>(db[i], db[i], dn[i]);
            mul_v<V>(dn[i], dn[i], wi);
            s1 += sum_v<V>(dn[i]);
            mul_v<V>(n, dn[i], xh[i]);
            s2 += sum_v<V>(n);
            if constexpr (GATED) store<T, V>(a.dgate, r * a.C + c + i * LANES * V, gt[i]);
        }
        const float minus_s1[1] = {-lanes_sum<LANES>(s1) * inv}, minus_s2[1] = {-lanes_sum<LANES>(s2) * inv};
        if constexpr (kRing) fetch(d, r + D * stride);        // (the slots have been read: the sums depend on them)
        if (!in) return;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (lane + i * LANES >= nvec) continue;
            add_v<V>(dn[i], dn[i], minus_s1);
            fma_v<V>(dn[i], xh[i], minus_s2, dn[i]);
            mul_v<V>(dn[i], dn[i], scale);
            store<T, V>(a.dx, r * a.C + c + i * LANES * V, dn[i]);
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d, (blockIdx.x + (int64_t)d * gridDim.x) * rsubs + rs);
    for (int64_t base = (int64_t)blockIdx.x * rsubs; base < a.N; base += D * stride)
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (base + d * stride < a.N) row(d, base + d * stride + rs);      // (the same for a whole block)
    if (!on || !a.dw) return;
    float* out = a.part + ((int64_t)blockIdx.x * rsubs + rs) * 2 * a.C + c;
#pragma unroll
    for (int i = 0; i < I; ++i)
        if (lane + i * LANES < nvec)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                out[i * LANES * V + j] = dw[i][j];
                out[a.C + i * LANES * V + j] = db[i][j];
            }
}

// dw and db: the sum of `parts` rows of (dw[C], db[C]) for 32 of the 2 C
// columns, in a fixed order, by 1024 threads.
__device__ __forceinline__ void sum_parts(const Args& a, int block) {
    __shared__ float sh[32][33];
    const int col = block * 32 + threadIdx.x % 32, r0 = threadIdx.x / 32;
    float s = 0.f;
    if (col < 2 * a.C) {
        const float* p = a.part + col;
#pragma unroll 8
        for (int r = r0; r < a.parts; r += 32) s += p[(int64_t)r * 2 * a.C];
    }
    sh[r0][threadIdx.x % 32] = s;
    __syncthreads();
    s = lanes_sum<32>(sh[threadIdx.x % 32][r0]);
    const int c = block * 32 + r0;
    if (threadIdx.x % 32 == 0 && c < 2 * a.C) {
        float& sum = c < a.C ? a.dw[c] : a.db[c - a.C];
        sum = a.add ? sum + s : s;
    }
}
__global__ void __launch_bounds__(1024) gn_sum_parts(const Args a) { sum_parts(a, blockIdx.x); }

// ----------------------------------------------------------- sample form ---
//
// A block takes every chunks-th part of a sample's positions and up to 256
// vectors of its channels: thread = (vector column, row lane).  The blocks of
// a sample so read one window of memory together: 8 x 4096 x 768 fp32 applies
// the backward pass in 38.2 us, 41.1 with a contiguous range for each block.
// Where the partial results of all samples would take over kPartBytes, some
// samples at a time go through all passes, so that a call's workspace does not
// grow with their number, and the passes find each other's results in L2.

struct Tile {
    int n, chunk, colv, rl, rows;             // rows: row lanes
    int count;                                // positions of this thread: first, first + step, ...
    int64_t first, step;                      // (counted over all samples)
    bool on;
};
template <int V>
__device__ __forceinline__ Tile tile_of(const Args& a, bool backwards) {
    const int bx = blockIdx.x;
    Tile t;
    t.n = bx / a.chunks;
    t.chunk = bx % a.chunks;
    const int cv = a.C / V, width = min(cv - (int)blockIdx.y * kThreads, kThreads);
    t.rows = (int)blockDim.x / width;
    t.rl = threadIdx.x / width;
    t.colv = blockIdx.y * kThreads + threadIdx.x % width;
    t.on = t.rl < t.rows;
    const int64_t s0 = (int64_t)t.chunk * t.rows + t.rl;
    t.step = (int64_t)a.chunks * t.rows;
    t.first = (int64_t)t.n * a.S + s0;
    t.count = s0 < a.S ? (int)((a.S - s0 + t.step - 1) / t.step) : 0;
    if (backwards) {
        t.first += (t.count - 1) * t.step;
        t.step = -t.step;
    }
    return t;
}
// A thread's positions, B at a time, the next ones' loads out during the work
// on these; fewer than B at the end one by one.  fetch(row) takes the next
// position, work(rows, integral_constant<n>) the n next ones.
template <int B, typename Row, typename Fetch, typename Work>
__device__ __forceinline__ void walk(int count, Fetch&& fetch, Work&& work) {
    Row next[B], now[B];
    int left = count;
    if (left >= B)
#pragma unroll
        for (int k = 0; k < B; ++k) fetch(next[k]);
    while (left >= B) {
#pragma unroll
        for (int k = 0; k < B; ++k) now[k] = next[k];
        left -= B;
        if (left >= B)
#pragma unroll
            for (int k = 0; k < B; ++k) fetch(next[k]);
        work(now, std::integral_constant<int, B>{});
    }
    if constexpr (B > 1) {
#pragma unroll
        for (int k = 0; k < B - 1; ++k)
            if (k < left) fetch(now[k]);
#pragma unroll 1
        for (int k = 0; k < left; ++k) {
            work(now, std::integral_constant<int, 1>{});
#pragma unroll
            for (int i = 0; i + 1 < B; ++i) now[i] = now[i + 1];
        }
    }
}
// The vectors of one position (those that there are), and where they come from.
template <typename T, int V, bool WITH_DY, bool GATED>
struct Row {
    Pack<T, V> x, dy, gate;
};
template <typename T, int V, bool WITH_DY, bool GATED, bool LAST>
struct Source {
    const T *x, *dy, *gate;
    int64_t sx, sd, sg;
    __device__ __forceinline__ Source(const Args& a, const Tile& t) {
        const int64_t c = (int64_t)t.colv * V;
        x = reinterpret_cast<const T*>(a.x) + t.first * a.ldx + c;
        sx = t.step * a.ldx;
        if constexpr (WITH_DY) {
            dy = reinterpret_cast<const T*>(a.dy) + t.first * a.ldy + c;
            sd = t.step * a.ldy;
        }
        if constexpr (GATED) {
            gate = reinterpret_cast<const T*>(a.gate) + t.first * a.ldg + c;
            sg = t.step * a.ldg;
        }
    }
    __device__ __forceinline__ void operator()(Row<T, V, WITH_DY, GATED>& r) {
        r.x = load<T, V, LAST>(x, 0);
        x += sx;
        if constexpr (WITH_DY) {
            r.dy = load<T, V, LAST>(dy, 0);
            dy += sd;
        }
        if constexpr (GATED) {
            r.gate = load<T, V, LAST>(gate, 0);
            gate += sg;
        }
    }
};

// (count, mean, sum of squared deviations) of two sets joined
__device__ __forceinline__ void join(float& n, float& m, float& q, float n2, float m2, float q2) {
    const float t = n + n2;
    if (n2 == 0.f) return;
    const float d = m2 - m, f = n2 / t;
    m = fmaf(d, f, m);
    q += q2 + d * (n * f) * d;                                // (the first set: 0 whatever d, whose square may overflow)
    n = t;
}

// Statistics of a block's part of every group: per channel first, from sums
// over a few positions at a time.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 3) gn_stats(const Args a) {
    __shared__ float sh_m[V * kThreads], sh_q[V * kThreads], sh_n[kThreads];      // [row lane][channel of the block]
    const Tile t = tile_of<V>(a, false);
    const int width = min(a.C / V - (int)blockIdx.y * kThreads, kThreads);
    float n = 0.f, m[V], q[V];
#pragma unroll
    for (int j = 0; j < V; ++j) m[j] = q[j] = 0.f;
    if (t.on)
        walk<4, Row<T, V, false, false>>(t.count, Source<T, V, false, false, false>(a, t), [&](auto& row, auto batch) {
            constexpr int B = decltype(batch)::value;
            const float f = (float)B / (n + (float)B);
            const float inv[1] = {1.f / (float)B}, minus[1] = {-1.f}, part[1] = {f}, both[1] = {n * f};
            float x[V], sum[V], sq[V], d[V];
#pragma unroll
            for (int k = 0; k < B; ++k) {
                unpack<T, V>(row[k].x, x);
                if (k == 0)
#pragma unroll
                    for (int j = 0; j < V; ++j) sum[j] = x[j];
                else
                    add_v<V>(sum, sum, x);
            }
            if (B > 1) mul_v<V>(sum, sum, inv);
#pragma unroll
            for (int k = 0; k < B; ++k) {
                unpack<T, V>(row[k].x, x);
                fma_v<V>(d, sum, minus, x);
                if (k == 0)
                    mul_v<V>(sq, d, d);
                else
                    fma_v<V>(sq, d, d, sq);
            }
            // joined with the positions before
            fma_v<V>(d, m, minus, sum);
            fma_v<V>(m, d, part, m);
            float e[V];
            mul_v<V>(e, d, both);
            fma_v<V>(sq, e, d, sq);
            add_v<V>(q, q, sq);
            n += (float)B;
        });
    if (t.on) {
        const int at = t.rl * width + (t.colv - (int)blockIdx.y * kThreads);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            sh_m[at * V + j] = m[j];
            sh_q[at * V + j] = q[j];
        }
        if (at % width == 0) sh_n[t.rl] = n;
    }
    __syncthreads();
    // one warp a group: its channels in every row lane
    const int c0 = (int)blockIdx.y * kThreads * V, c1 = c0 + width * V;
    const int lane = threadIdx.x % 32;
    const bool all = gridDim.y == 1;
    const int g0 = all ? 0 : c0 / a.D, g1 = all ? a.G : (c1 - 1) / a.D + 1;
    for (int g = g0 + threadIdx.x / 32; g < g1; g += (int)blockDim.x / 32) {
        float gn = 0.f, gm = 0.f, gq = 0.f;
        const int lo = max(g * a.D, c0) - c0, hi = min((g + 1) * a.D, c1) - c0;
        for (int e = lane; e < (hi - lo) * t.rows; e += 32) {
            const int row = e / (hi - lo), at = row * width * V + lo + e % (hi - lo);
            join(gn, gm, gq, sh_n[row], sh_m[at], sh_q[at]);
        }
        for (int d = 16; d > 0; d >>= 1) {
            const float n2 = __shfl_down_sync(0xffffffffu, gn, d), m2 = __shfl_down_sync(0xffffffffu, gm, d),
                        q2 = __shfl_down_sync(0xffffffffu, gq, d);
            join(gn, gm, gq, n2, m2, q2);
        }
        if (lane == 0) {
            const int column = (int)blockIdx.y - g * a.D / (kThreads * V);    // among the blocks with channels of the group
            const int64_t e = ((int64_t)t.n * a.G + g) * a.parts + (int64_t)column * a.chunks + t.chunk;
            reinterpret_cast<float4*>(a.part)[e] = make_float4(gn, gm, gq, 0.f);
        }
    }
}

// One warp a (sample, group): joins its parts, those of every block of
// `columns` channels that the group reaches into.
__global__ void __launch_bounds__(kThreads) gn_join_stats(const Args a, int columns) {
    const int64_t p = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    if (p >= a.N * a.G) return;
    const int lane = threadIdx.x % 32;
    int parts = a.chunks;
    if (a.parts > a.chunks) {
        const int c0 = (int)((uint32_t)p % (uint32_t)a.G) * a.D;              // (N G is below 2^31)
        parts *= (c0 + a.D - 1) / columns - c0 / columns + 1;
    }
    float n = 0.f, m = 0.f, q = 0.f;
#pragma unroll 4
    for (int e = lane; e < parts; e += 32) {
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

// A statistic of a thread's channels: one value where the vector lies in one
// group (WHOLE), else one a channel.
template <int V, bool WHOLE>
struct Stat {
    float v[WHOLE ? 1 : V];
    __device__ __forceinline__ void negate() {
#pragma unroll
        for (int j = 0; j < (WHOLE ? 1 : V); ++j) v[j] = -v[j];
    }
    __device__ __forceinline__ void read(const float* p, int64_t row, int c, int D, int step) {
#pragma unroll
        for (int j = 0; j < (WHOLE ? 1 : V); ++j) v[j] = p[(row + (c + j) / D) * step];
    }
};

template <typename T, int V, bool WHOLE, bool GATED>
__global__ void __launch_bounds__(kThreads, 3) gn_apply(const Args a) {
    const Tile t = tile_of<V>(a, true);
    if (!t.on) return;
    const int c = t.colv * V;
    float w[V], b[V];
    load_w<T, V>(a.w, a.w_f32, c, 1.f, w);
    load_w<T, V>(a.b, a.w_f32, c, 0.f, b);
    Stat<V, WHOLE> mean, rstd;
    mean.read(a.mean, (int64_t)t.n * a.G, c, a.D, 1);
    rstd.read(a.rstd, (int64_t)t.n * a.G, c, a.D, 1);
    mul_v<V>(w, w, rstd.v);
    mean.negate();
    T* y = reinterpret_cast<T*>(a.y) + t.first * a.C + c;
    walk<GATED ? 2 : 4, Row<T, V, false, GATED>>(
        t.count, Source<T, V, false, GATED, true>(a, t), [&](auto& row, auto batch) {
#pragma unroll
            for (int k = 0; k < decltype(batch)::value; ++k) {
                float f[V], g[V];
                unpack<T, V>(row[k].x, f);
                if constexpr (GATED) unpack<T, V>(row[k].gate, g);
                add_v<V>(f, f, mean.v);
                fma_v<V>(f, f, w, b);
                finish<V, GATED>(f, g, a.act);
                store<T, V>(y, 0, f);
                y += t.step * a.C;
            }
        });
}

// xh, dn and dgate of one vector (mean: negated)
template <typename T, int V, bool WHOLE, bool GATED>
__device__ __forceinline__ void grad_of(const Args& a, const Row<T, V, true, GATED>& row, const Stat<V, WHOLE>& mean,
                                        const Stat<V, WHOLE>& rstd, const float (&w)[V], const float (&b)[V],
                                        float (&xh)[V], float (&dn)[V], float (&dg)[V]) {
    float n[V];
    unpack<T, V>(row.x, xh);
    unpack<T, V>(row.dy, dn);
    if constexpr (GATED) unpack<T, V>(row.gate, dg);
    add_v<V>(xh, xh, mean.v);
    mul_v<V>(xh, xh, rstd.v);
    fma_v<V>(n, xh, w, b);
    start<V, GATED>(n, dn, dg, a.act);
}

// First backward pass: the sums of dn xh and dn over the chunk's positions,
// by channel: part[(sample, chunk)][2][C].
template <typename T, int V, bool WHOLE, bool GATED>
__global__ void __launch_bounds__(kThreads, WHOLE || V < 8 ? 3 : 2) gn_grad_sums(const Args a) {
    __shared__ float sh[2][kThreads * V];
    const Tile t = tile_of<V>(a, false);
    const int width = min(a.C / V - (int)blockIdx.y * kThreads, kThreads);
    float s1[V], s2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) s1[j] = s2[j] = 0.f;
    const int c = t.colv * V;
    if (t.on) {
        float w[V], b[V];
        load_w<T, V>(a.w, a.w_f32, c, 1.f, w);
        load_w<T, V>(a.b, a.w_f32, c, 0.f, b);
        Stat<V, WHOLE> mean, rstd;
        mean.read(a.mean, (int64_t)t.n * a.G, c, a.D, 1);
        rstd.read(a.rstd, (int64_t)t.n * a.G, c, a.D, 1);
        mean.negate();
        walk<GATED ? 1 : 2, Row<T, V, true, GATED>>(
            t.count, Source<T, V, true, GATED, false>(a, t), [&](auto& row, auto batch) {
#pragma unroll
                for (int k = 0; k < decltype(batch)::value; ++k) {
                    float xh[V], dn[V], dg[V];
                    grad_of<T, V, WHOLE, GATED>(a, row[k], mean, rstd, w, b, xh, dn, dg);
                    fma_v<V>(s1, dn, xh, s1);
                    add_v<V>(s2, s2, dn);
                }
            });
#pragma unroll
        for (int j = 0; j < V; ++j) {
            sh[0][(t.rl * width + t.colv - (int)blockIdx.y * kThreads) * V + j] = s1[j];
            sh[1][(t.rl * width + t.colv - (int)blockIdx.y * kThreads) * V + j] = s2[j];
        }
    }
    __syncthreads();
    float* out = a.part + (int64_t)blockIdx.x * 2 * a.C + (int64_t)blockIdx.y * kThreads * V;
    for (int e = threadIdx.x; e < width * V; e += (int)blockDim.x) {
        float x = 0.f, y = 0.f;
        for (int r = 0; r < t.rows; ++r) {
            x += sh[0][r * width * V + e];
            y += sh[1][r * width * V + e];
        }
        out[e] = x;
        out[a.C + e] = y;
    }
}

// One block a (sample, group): mean(dn w) and mean(dn w xh); the blocks behind
// them sum dw and db.
template <typename T>
__global__ void __launch_bounds__(1024) gn_join_sums(const Args a) {
    if (blockIdx.x >= a.N * a.G) return sum_parts(a, (int)(blockIdx.x - a.N * a.G));
    __shared__ float sh[2][32];
    const int64_t p = blockIdx.x, n = p / a.G;
    const int c0 = (int)(p % a.G) * a.D;
    float s1 = 0.f, s2 = 0.f;
    // (chunk, channel) in order of memory
#pragma unroll 4
    for (int e = threadIdx.x; e < a.D * a.chunks; e += (int)blockDim.x) {
        const int k = e / a.D, c = c0 + e % a.D;
        float w[1];
        load_w<T, 1>(a.w, a.w_f32, c, 1.f, w);
        const float* src = a.part + (n * a.chunks + k) * 2 * a.C + c;
        s1 = fmaf(src[0], w[0], s1);
        s2 = fmaf(src[a.C], w[0], s2);
    }
    s1 = lanes_sum<32>(s1);
    s2 = lanes_sum<32>(s2);
    if (threadIdx.x % 32 == 0) {
        sh[0][threadIdx.x / 32] = s1;
        sh[1][threadIdx.x / 32] = s2;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const bool in = threadIdx.x < blockDim.x / 32;
        s1 = lanes_sum<32>(in ? sh[0][threadIdx.x] : 0.f);
        s2 = lanes_sum<32>(in ? sh[1][threadIdx.x] : 0.f);
        if (threadIdx.x == 0) {
            const float inv = 1.f / ((float)a.S * (float)a.D);
            a.sums[2 * p] = s2 * inv;
            a.sums[2 * p + 1] = s1 * inv;
        }
    }
}

template <typename T, int V, bool WHOLE, bool GATED>
__global__ void __launch_bounds__(kThreads, WHOLE || V < 8 ? 3 : 2) gn_grad_apply(const Args a) {
    const Tile t = tile_of<V>(a, true);
    if (!t.on) return;
    const int c = t.colv * V;
    float w[V], b[V];
    load_w<T, V>(a.w, a.w_f32, c, 1.f, w);
    load_w<T, V>(a.b, a.w_f32, c, 0.f, b);
    Stat<V, WHOLE> mean, rstd, m1, m2;
    mean.read(a.mean, (int64_t)t.n * a.G, c, a.D, 1);
    rstd.read(a.rstd, (int64_t)t.n * a.G, c, a.D, 1);
    m1.read(a.sums, (int64_t)t.n * a.G, c, a.D, 2);
    m2.read(a.sums + 1, (int64_t)t.n * a.G, c, a.D, 2);
    mean.negate();
    m1.negate();
    m2.negate();
    T *dx = reinterpret_cast<T*>(a.dx) + t.first * a.C + c, *dgate = reinterpret_cast<T*>(a.dgate) + t.first * a.C + c;
    walk<GATED ? 1 : 2, Row<T, V, true, GATED>>(
        t.count, Source<T, V, true, GATED, true>(a, t), [&](auto& row, auto batch) {
#pragma unroll
            for (int k = 0; k < decltype(batch)::value; ++k) {
                float xh[V], dn[V], dg[V];
                grad_of<T, V, WHOLE, GATED>(a, row[k], mean, rstd, w, b, xh, dn, dg);
                if constexpr (GATED) {
                    store<T, V>(dgate, 0, dg);
                    dgate += t.step * a.C;
                }
                fma_v<V>(dn, dn, w, m1.v);
                fma_v<V>(dn, xh, m2.v, dn);
                mul_v<V>(dn, dn, rstd.v);
                store<T, V>(dx, 0, dn);
                dx += t.step * a.C;
            }
        });
}

// ------------------------------------------------------------------ host ---

int fail(int status, const std::string& msg) {
    set_last_error(msg.c_str());
    return status;
}

// Blocks of the token form at most, all resident: they walk down the rows.
// (B200's number of SMs here and in chunks_of, so that a workspace's size does
// not depend on the current device.)
constexpr int64_t kTokenBlocks = 148 * 3;

// Threads of the sample form's blocks: whole rows of vector columns.
int sample_threads(int64_t S, int64_t C, int V) {
    const int64_t cv = C / V > 0 ? C / V : 1, width = cv < kThreads ? cv : kThreads;
    int64_t rows = kThreads / width;
    if (rows > S) rows = S;
    return (int)((width * rows + 31) / 32 * 32);
}
// Samples are cut so that all blocks are resident at once where there are few
// samples (768 threads an SM; twice as many chunks: 35 us instead of 30 for the
// statistics of 16 x 4095 x 760 fp16), but no finer than 16384 values.
int64_t chunks_of(int64_t N, int64_t S, int64_t C, int V) {
    const int64_t cols = (C / V + kThreads - 1) / kThreads > 0 ? (C / V + kThreads - 1) / kThreads : 1;
    int64_t want = 148 * (768 / sample_threads(S, C, V)) / ((N > 0 ? N : 1) * cols);
    const int64_t most = S * C / 16384;
    if (want > most) want = most;
    if (want > S) want = S;
    return want > 1 ? want : 1;
}
constexpr int64_t kPartBytes = 64 << 20;      // half of L2

int64_t columns_of(int64_t C, int V) { return (C / V + kThreads - 1) / kThreads; }
// Blocks of columns with channels of one group, at most.
int64_t spread_of(int64_t C, int64_t G, int V) {
    const int64_t width = kThreads * V, most = (C / G + width - 2) / width + 1, cols = columns_of(C, V);
    return most < cols ? most : cols;
}
// Samples that go through the sample form's passes together.
int64_t samples_at_once(int64_t N, int64_t S, int64_t C, int64_t G, int V, bool back) {
    const int64_t chunks = chunks_of(N, S, C, V);
    const int64_t bytes = back ? chunks * 2 * C * 4 + G * 8 : chunks * spread_of(C, G, V) * G * 16 + G * 8;
    const int64_t most = kPartBytes / bytes > 1 ? kPartBytes / bytes : 1, times = (N + most - 1) / most;
    return times > 1 ? (N + times - 1) / times : N;
}

// Lanes and vectors a lane of the token form for groups of nvec vectors of V
// elements; 0 lanes: too wide for it (over 512 channels, or 256 one by one).
void token_shape(int64_t nvec, int V, int& lanes, int& per) {
    lanes = 1;
    while (lanes < 32 && lanes < nvec) lanes *= 2;
    per = 1;
    while (per * lanes < nvec) per *= 2;
    if (per > (V == 8 ? 2 : V == 4 ? 4 : 8)) lanes = 0;
}

struct TokenGrid {
    int gsubs, rsubs, threads;
    unsigned gx, gy;
};
// Blocks of whole rows where the groups of one fit, so that a block's loads
// are contiguous; as many as fill the GPU, or fewer where rows run out.
TokenGrid token_grid(int64_t N, int64_t G, int lanes, int rows_at_once) {
    TokenGrid t;
    const int subs = kThreads / lanes;
    t.gsubs = (int)(G < subs ? G : subs);
    t.rsubs = subs / t.gsubs;
    if (t.rsubs > N) t.rsubs = (int)N;
    t.threads = (t.gsubs * t.rsubs * lanes + 31) / 32 * 32;
    t.gy = (unsigned)((G + t.gsubs - 1) / t.gsubs);
    const int64_t most = kTokenBlocks / t.gy > 1 ? kTokenBlocks / t.gy : 1;
    const int64_t rows = (N + t.rsubs * rows_at_once - 1) / (t.rsubs * rows_at_once);
    t.gx = (unsigned)(rows < most ? rows : most);
    return t;
}

template <typename T, int V, int I, int LANES>
void token_launch(const Args& a, const TokenGrid& t, bool back, cudaStream_t s) {
    const dim3 grid(t.gx, t.gy);
    if (back)
        a.gate ? gn_token_backward<T, V, I, LANES, true><<<grid, t.threads, 0, s>>>(a, t.gsubs, t.rsubs)
               : gn_token_backward<T, V, I, LANES, false><<<grid, t.threads, 0, s>>>(a, t.gsubs, t.rsubs);
    else
        a.gate ? gn_token_forward<T, V, I, LANES, true><<<grid, t.threads, 0, s>>>(a, t.gsubs, t.rsubs)
               : gn_token_forward<T, V, I, LANES, false><<<grid, t.threads, 0, s>>>(a, t.gsubs, t.rsubs);
}

// (the rows that a sub-warp has in flight, as the kernels choose them)
int rows_at_once(int per, bool back) { return !back && per == 1 ? 2 : 1; }

template <typename T, int V>
void token(Args a, int lanes, int per, bool back, cudaStream_t s) {
    const TokenGrid t = token_grid(a.N, a.G, lanes, rows_at_once(per, back));
    a.parts = (int)t.gx * t.rsubs;
    if (per == 1) {
        switch (lanes) {
            case 1: token_launch<T, V, 1, 1>(a, t, back, s); break;
            case 2: token_launch<T, V, 1, 2>(a, t, back, s); break;
            case 4: token_launch<T, V, 1, 4>(a, t, back, s); break;
            case 8: token_launch<T, V, 1, 8>(a, t, back, s); break;
            case 16: token_launch<T, V, 1, 16>(a, t, back, s); break;
            default: token_launch<T, V, 1, 32>(a, t, back, s); break;
        }
    } else if (per == 2) {
        token_launch<T, V, 2, 32>(a, t, back, s);
    } else if constexpr (V < 8) {
        if (per == 4) {
            token_launch<T, V, 4, 32>(a, t, back, s);
        } else if constexpr (V == 1) {
            token_launch<T, V, 8, 32>(a, t, back, s);
        }
    }
    if (back && a.dw) gn_sum_parts<<<(unsigned)((2 * a.C + 31) / 32), 1024, 0, s>>>(a);
}

template <typename T, int V, bool WHOLE, bool GATED>
void sample_of(Args a, bool back, cudaStream_t s) {
    const unsigned cols = (unsigned)columns_of(a.C, V);
    a.chunks = (int)chunks_of(a.N, a.S, a.C, V);
    const int threads = sample_threads(a.S, a.C, V);
    const int64_t all = a.N, step = samples_at_once(a.N, a.S, a.C, a.G, V, back);
    auto on = [](auto& p, int64_t by) {
        if (p) p = (std::remove_reference_t<decltype(p)>)((const uint8_t*)p + by);
    };
    for (int64_t n0 = 0; n0 < all; n0 += step) {
        a.N = step < all - n0 ? step : all - n0;
        const dim3 grid((unsigned)(a.N * a.chunks), cols);
        if (!back) {
            a.parts = (int)(spread_of(a.C, a.G, V) * a.chunks);
            gn_stats<T, V><<<grid, threads, 0, s>>>(a);
            gn_join_stats<<<(unsigned)((a.N * a.G + 7) / 8), kThreads, 0, s>>>(a, kThreads * V);
            gn_apply<T, V, WHOLE, GATED><<<grid, threads, 0, s>>>(a);
        } else {
            a.parts = (int)(a.N * a.chunks);
            a.add = n0 > 0;
            gn_grad_sums<T, V, WHOLE, GATED><<<grid, threads, 0, s>>>(a);
            const int64_t values = (int64_t)a.D * a.chunks;
            if (a.dw)
                gn_join_sums<T><<<(unsigned)(a.N * a.G + (2 * a.C + 31) / 32), 1024, 0, s>>>(a);
            else
                gn_join_sums<T><<<(unsigned)(a.N * a.G), values > 256 ? 1024 : 256, 0, s>>>(a);
            gn_grad_apply<T, V, WHOLE, GATED><<<grid, threads, 0, s>>>(a);
        }
        const int64_t rows = step * a.S, es = sizeof(T);
        on(a.x, rows * a.ldx * es);
        on(a.gate, rows * a.ldg * es);
        on(a.dy, rows * a.ldy * es);
        on(a.y, rows * a.C * es);
        on(a.dx, rows * a.C * es);
        on(a.dgate, rows * a.C * es);
        if (a.keep || back) {                                 // (else they lie in the workspace)
            on(a.mean, step * a.G * 4);
            on(a.rstd, step * a.G * 4);
        }
    }
}

template <typename T, int V>
void sample(const Args& a, bool back, cudaStream_t s) {
    if constexpr (V > 1) {
        if (a.D % V) return a.gate ? sample_of<T, V, false, true>(a, back, s) : sample_of<T, V, false, false>(a, back, s);
    }
    a.gate ? sample_of<T, V, true, true>(a, back, s) : sample_of<T, V, true, false>(a, back, s);
}

template <typename T, int V>
void run(const Args& a, bool back, cudaStream_t s) {
    int lanes = 0, per = 0;
    if (a.S == 1 && a.D % V == 0) token_shape(a.D / V, V, lanes, per);
    if (lanes > 0)
        token<T, V>(a, lanes, per, back, s);
    else
        sample<T, V>(a, back, s);
}

// Vectors need rows that are whole vectors; the token form whole groups too.
bool use_vectors(const Args& a, int V, bool rows_aligned) {
    if (!rows_aligned || a.C % V) return false;
    if (a.S == 1 && a.D % V) {
        // groups that are no whole vectors: element by element in the token
        // form (one pass) unless they are too wide for it
        int lanes, per;
        token_shape(a.D, 1, lanes, per);
        return lanes == 0;
    }
    return true;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int64_t pad256(int64_t b) { return (b + 255) / 256 * 256; }

int vec_of(int dtype) { return dtype == FFTCONV_F32 ? 4 : 8; }

// Workspace of a call with vectors of V elements: the sample form's sums (or
// mean and rstd where the caller keeps none), then partial results.  Sizes of 0
// where a form has none.
struct Space {
    int64_t sums, part;
};
Space space_of(int64_t N, int64_t S, int64_t C, int64_t G, int V, bool back) {
    const int64_t D = C / G;
    int lanes = 0, per = 0;
    if (S == 1 && D % V == 0) token_shape(D / V, V, lanes, per);
    if (lanes > 0) {
        // rows of the token form's blocks' sub-warps
        const TokenGrid t = token_grid(N, G, lanes, rows_at_once(per, back));
        return {0, back ? pad256((int64_t)t.gx * t.rsubs * 2 * C * 4) : 0};
    }
    const int64_t n = samples_at_once(N, S, C, G, V, back), chunks = chunks_of(N, S, C, V);
    return back ? Space{pad256(n * G * 8), pad256(n * chunks * 2 * C * 4)}
                : Space{2 * pad256(n * G * 4), pad256(n * chunks * spread_of(C, G, V) * G * 16)};
}

// Whether the token form's blocks of groups are within a grid's second extent
// (8.4 M channels at least; the sample form's columns always are, see check).
bool grid_fits(int64_t N, int64_t S, int64_t C, int64_t G, int V) {
    const int64_t D = C / G;
    int lanes = 0, per = 0;
    if (S == 1 && D % V == 0) token_shape(D / V, V, lanes, per);
    return lanes == 0 || token_grid(N, G, lanes, 1).gy <= 65535;
}

// The largest of the vector widths that a call may take (which depends on
// strides and on the type).
size_t workspace_bytes(int64_t N, int64_t S, int64_t C, int64_t G, bool back) {
    if (N == 0 || S == 0 || C == 0) return 0;
    Args a{};
    a.S = S;
    a.C = (int)C;
    a.D = (int)(C / G);
    int64_t most = 0;
    for (int V : {1, 4, 8}) {
        if (V > 1 && !use_vectors(a, V, true)) continue;
        const Space w = space_of(N, S, C, G, V, back);
        if (w.sums + w.part > most) most = w.sums + w.part;
    }
    return (size_t)most;
}

int check(int64_t N, int64_t S, int64_t C, int64_t G, int dtype, int wdtype, int act, bool affine) {
    if (N < 0 || S < 0 || C <= 0 || G <= 0) return fail(FFTCONV_ERR_INVALID_ARG, "N, S, C or G out of range");
    if (C % G) return fail(FFTCONV_ERR_INVALID_ARG, "G must divide C");
    if (dtype != FFTCONV_F32 && dtype != FFTCONV_F16 && dtype != FFTCONV_BF16)
        return fail(FFTCONV_ERR_INVALID_ARG, "unknown dtype");
    if (affine && wdtype != dtype && wdtype != FFTCONV_F32)
        return fail(FFTCONV_ERR_INVALID_ARG, "weight and bias must have x's type or fp32");
    if (act < FFTCONV_ACT_NONE || act > FFTCONV_ACT_SIGMOID) return fail(FFTCONV_ERR_INVALID_ARG, "unknown activation");
    if (C > 65535 * kThreads || (double)N * (double)G >= 2147483647.0 || (double)N + (double)C >= 2147483647.0 - 444.0)
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
    const int V = vec_of(dtype);
    const bool vec = use_vectors(a, V, rows == 1 || (ld_x % V == 0 && (!gate || ld_gate % V == 0)));
    if (!grid_fits(N, S, C, G, vec ? V : 1)) return fail(FFTCONV_ERR_UNSUPPORTED, "too many groups for one launch");
    a.mean = mean;
    a.rstd = rstd;
    a.keep = mean != nullptr;
    const Space space = space_of(N, S, C, G, vec ? V : 1, false);
    a.part = (float*)((uint8_t*)workspace + space.sums);
    if (!mean && space.sums) {
        a.mean = (float*)workspace;
        a.rstd = (float*)((uint8_t*)workspace + space.sums / 2);
    }
    (void)cudaGetLastError();                                 // (an earlier call's error is not this one's)
    dispatch(dtype, vec, [&](auto* t, auto v) {
        using T = std::remove_pointer_t<decltype(t)>;
        run<T, decltype(v)::value>(a, false, (cudaStream_t)stream);
    });
    const cudaError_t e = cudaGetLastError();
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
    const int V = vec_of(dtype);
    const bool vec =
        use_vectors(a, V, rows == 1 || (ld_x % V == 0 && ld_dy % V == 0 && (!gate || ld_gate % V == 0)));
    if (!grid_fits(N, S, C, G, vec ? V : 1)) return fail(FFTCONV_ERR_UNSUPPORTED, "too many groups for one launch");
    a.sums = (float*)workspace;
    a.part = (float*)((uint8_t*)workspace + space_of(N, S, C, G, vec ? V : 1, true).sums);
    (void)cudaGetLastError();                                 // (an earlier call's error is not this one's)
    dispatch(dtype, vec, [&](auto* t, auto v) {
        using T = std::remove_pointer_t<decltype(t)>;
        run<T, decltype(v)::value>(a, true, s);
    });
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? FFTCONV_OK
                            : fail(FFTCONV_ERR_CUDA, std::string("group norm backward launch: ") + cudaGetErrorString(e));
}

}  // extern "C"
