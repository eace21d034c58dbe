// linear_attention_step.cu -- the single-token form of linear attention:
//     S <- g S + k v^T (in place),   o = scale * q S
// for each row and head of a batch.  The state (K x V fp32) is read and
// written once and dominates: 8 K V bytes against 2 (2 K + 2 V) for the token.
// One CTA takes one state; every thread owns four columns of a few rows, so a
// warp reads whole 512-byte rows in 16-byte pieces, and the sums over K are
// joined once through shared memory.  Four rows a thread in flight and six
// CTAs an SM, loads and stores marked as read once: 89 us for 250 x 16 states
// of 128 x 128 on B200 (5.8 TB/s, 90% of a copy's rate), against 101 us with
// eight rows and four CTAs and 93 us without the marks; six CTAs leave 40
// registers a thread, and 40 bytes are spilled.
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
    const void *q, *k, *v;
    const float* log_decay;
    float* state;
    const int32_t* slots;
    void* o;
    int64_t qb, qh, kb, kh, vb, vh;
    int64_t pool;
    int H, q_div, k_div, v_div, K, V;
    float scale;
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// LPR lanes (a power of two >= V / 4) hold one row of the state.
template <typename T, int LPR>
__global__ void __launch_bounds__(kThreads, 6) la_step_kernel(const Args a) {
    constexpr int kRows = kThreads / LPR;                     // rows in flight together
    __shared__ float qs[128], ks[128];
    __shared__ float4 part[kThreads];
    const int tid = threadIdx.x, h = blockIdx.x % a.H;
    const int64_t b = blockIdx.x / a.H;
    T* o = reinterpret_cast<T*>(a.o) + (b * a.H + h) * a.V;
    const int64_t slot = a.slots ? a.slots[b] : b;
    const bool valid = slot >= 0 && slot < a.pool;
    const T* q = reinterpret_cast<const T*>(a.q) + b * a.qb + (h / a.q_div) * a.qh;
    const T* k = reinterpret_cast<const T*>(a.k) + b * a.kb + (h / a.k_div) * a.kh;
    const T* v = reinterpret_cast<const T*>(a.v) + b * a.vb + (h / a.v_div) * a.vh;
    const int col = tid % LPR * 4, row0 = tid / LPR;
    const bool live = valid && col < a.V;
    float4* s = reinterpret_cast<float4*>(a.state + ((valid ? slot : 0) * a.H + h) * a.K * a.V + col);
    const int64_t step = a.V / 4;                             // float4s of a row
    constexpr int kAhead = 4;
    float4 x[kAhead];
    if (live) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (row0 + i * kRows < a.K) x[i] = __ldcs(&s[(row0 + i * kRows) * step]);
    }
    if (a.slots) {
        // (while the state's first rows are on their way)
        int idle = !valid;
        for (int64_t i = tid; i < b; i += kThreads) idle |= a.slots[i] == (int32_t)slot;
        if (__syncthreads_or(idle)) {
            if (tid < a.V) o[tid] = from_f<T>(0.f);
            return;
        }
    }
    if (tid < a.K) {
        qs[tid] = to_f(q[tid]) * a.scale;
        ks[tid] = to_f(k[tid]);
    }
    float4 vv = make_float4(0.f, 0.f, 0.f, 0.f), acc = vv;
    if (live) vv = make_float4(to_f(v[col]), to_f(v[col + 1]), to_f(v[col + 2]), to_f(v[col + 3]));
    const float g = expf(a.log_decay[h]);
    __syncthreads();
    if (live) {
        for (int r = row0; r < a.K; r += kAhead * kRows) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int row = r + i * kRows;
                if (row < a.K) {
                    const float kk = ks[row], qq = qs[row];
                    float4 y = x[i];
                    // the load of this slot's next row goes out before its use
                    if (row + kAhead * kRows < a.K) x[i] = __ldcs(&s[(row + kAhead * kRows) * step]);
                    y.x = fmaf(g, y.x, kk * vv.x);
                    y.y = fmaf(g, y.y, kk * vv.y);
                    y.z = fmaf(g, y.z, kk * vv.z);
                    y.w = fmaf(g, y.w, kk * vv.w);
                    __stcs(&s[row * step], y);
                    acc.x = fmaf(qq, y.x, acc.x);
                    acc.y = fmaf(qq, y.y, acc.y);
                    acc.z = fmaf(qq, y.z, acc.z);
                    acc.w = fmaf(qq, y.w, acc.w);
                }
            }
        }
    }
    part[tid] = acc;
    __syncthreads();
    if (tid < a.V) {
        const float* p = reinterpret_cast<const float*>(part) + tid;
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) sum += p[r * LPR * 4];
        o[tid] = from_f<T>(sum);
    }
}

int fail(int status, const std::string& msg) {
    set_last_error(msg.c_str());
    return status;
}

template <typename T>
void launch(const Args& a, unsigned ctas, cudaStream_t s) {
    const int lanes = a.V / 4;
    if (lanes > 16)
        la_step_kernel<T, 32><<<ctas, kThreads, 0, s>>>(a);
    else if (lanes > 8)
        la_step_kernel<T, 16><<<ctas, kThreads, 0, s>>>(a);
    else
        la_step_kernel<T, 8><<<ctas, kThreads, 0, s>>>(a);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

}  // namespace
}  // namespace fftconv

using namespace fftconv;

extern "C" int fftconv_linear_attention_step(const void* q, const void* k, const void* v, const float* log_decay,
                                             float* state, const int32_t* slots, void* o, int64_t B, int64_t pool,
                                             int64_t H, int64_t Hq, int64_t Hk, int64_t Hv, int64_t K, int64_t V,
                                             fftconv_dtype_t dtype, float scale, const int64_t* q_stride,
                                             const int64_t* k_stride, const int64_t* v_stride,
                                             fftconv_stream_t stream) {
    set_last_error("");
    if (B < 0 || pool < 0) return fail(FFTCONV_ERR_INVALID_ARG, "B or pool is negative");
    if (H <= 0 || Hq <= 0 || Hk <= 0 || Hv <= 0 || H % Hq || H % Hk || H % Hv)
        return fail(FFTCONV_ERR_INVALID_ARG, "Hq, Hk and Hv must be positive and divide H");
    if (dtype != FFTCONV_F16 && dtype != FFTCONV_BF16)
        return fail(dtype == FFTCONV_F32 ? FFTCONV_ERR_UNSUPPORTED : FFTCONV_ERR_INVALID_ARG,
                    "linear attention takes fp16 or bf16 tensors");
    if (K <= 0 || V <= 0) return fail(FFTCONV_ERR_INVALID_ARG, "K and V must be positive");
    if (K % 8 || V % 8 || K > 128 || V > 128)
        return fail(FFTCONV_ERR_UNSUPPORTED, "K and V must be multiples of 8 up to 128");
    if (!slots && pool != B) return fail(FFTCONV_ERR_INVALID_ARG, "without slots the pool has one state a row");
    if (pool >= (int64_t(1) << 31) || (double)B * (double)H >= 2147483647.0)
        return fail(FFTCONV_ERR_UNSUPPORTED, "too many rows or states");
    if (B == 0) return FFTCONV_OK;
    if (!q || !k || !v || !log_decay || !o || !q_stride || !k_stride || !v_stride || (!state && pool > 0))
        return fail(FFTCONV_ERR_INVALID_ARG, "q, k, v, log_decay, state, o and the strides must be non-NULL");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(state) || !aligned16(o))
        return fail(FFTCONV_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
    const int64_t* st[3] = {q_stride, k_stride, v_stride};
    const int64_t heads[3] = {Hq, Hk, Hv}, dims[3] = {K, K, V};
    const void* in[3] = {q, k, v};
    const int64_t states = pool * H * K * V * 4;
    for (int i = 0; i < 3; ++i) {
        if ((B > 1 && st[i][0] <= 0) || (heads[i] > 1 && st[i][1] <= 0))
            return fail(FFTCONV_ERR_INVALID_ARG, "strides must be positive");
        const int64_t span = ((B > 1 ? (B - 1) * st[i][0] : 0) + (heads[i] > 1 ? (heads[i] - 1) * st[i][1] : 0) + dims[i]) * 2;
        if (overlap(o, B * H * V * 2, in[i], span) || overlap(state, states, in[i], span))
            return fail(FFTCONV_ERR_INVALID_ARG, "o or state overlaps an input");
    }
    if (overlap(o, B * H * V * 2, state, states)) return fail(FFTCONV_ERR_INVALID_ARG, "o overlaps state");
    Args a{};
    a.q = q; a.k = k; a.v = v;
    a.log_decay = log_decay;
    a.state = state;
    a.slots = slots;
    a.o = o;
    a.qb = q_stride[0]; a.qh = q_stride[1];
    a.kb = k_stride[0]; a.kh = k_stride[1];
    a.vb = v_stride[0]; a.vh = v_stride[1];
    a.pool = pool;
    a.H = (int)H;
    a.q_div = (int)(H / Hq); a.k_div = (int)(H / Hk); a.v_div = (int)(H / Hv);
    a.K = (int)K; a.V = (int)V;
    a.scale = scale;
    cudaStream_t s = (cudaStream_t)stream;
    (void)cudaGetLastError();                                 // (an earlier call's error is not this one's)
    if (dtype == FFTCONV_F16)
        launch<__half>(a, (unsigned)(B * H), s);
    else
        launch<__nv_bfloat16>(a, (unsigned)(B * H), s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(FFTCONV_ERR_CUDA, std::string("linear attention step launch: ") + cudaGetErrorString(e));
    return FFTCONV_OK;
}
