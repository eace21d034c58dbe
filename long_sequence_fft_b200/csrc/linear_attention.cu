// linear_attention.cu -- causal linear attention with a decay for each head:
// the chunked prompt form on the tensor cores, forward and backward.
//
// Mathematics.  With g = exp(log_decay[h]), a query side x, a key side y and
// a value side z, the kernel evaluates over the tokens of one sequence, in
// either direction of time,
//
//     o_t = a sum_{s at or before t} g^|t-s| (x_t . y_s) z_s + (carry term)
//
// in chunks of 128 tokens: P = (x y^T) * a g^|i-j| inside the chunk (masked to
// its triangle), o = P z + g^(...) x C with the carried state C (key dim x
// value dim, fp32 in registers), and C <- g^n C + sum_j g^(...) y_j z_j^T.
// The forward pass is (x, y, z) = (q, k, v) forward in time.  The gradients
// are the same sums:
//     dq = (do, v, k) forward in time, carry = S^T
//     dk = (v, do, q), dv = (k, q, do) backward in time, carry = dS^T and dS,
// so the backward pass is one launch with three roles.
//
// What bounds it.  A chunk of 128/128 bf16 moves 128 KB (its share of the
// card's bandwidth: 5800 clocks of an SM) and takes five products of 128^3
// (520 clocks each at the dense rate); measured, 6000 to 6500 clocks.  At
// 64/64 it is 64 KB, 2900 clocks against 2950.  fp16 takes 8000 and 4100: the
// rows' and the keys' scales are found by warps that the products wait for.
// So the forward pass is at the memory's rate while every SM has a chunk; what
// is lost is the second reading of keys and values where few heads make a cut
// along time necessary, and the last wave (B200, 16 x 4096 tokens, 12 heads of
// 64/64, forward and backward: 330 us, of 172 for the bytes; 65536 tokens, 16
// heads of 128/128: 320 us, of 167; both at 1965 MHz, and a fifth more once
// seconds of it meet the power limit at 1490).  The chunk's length is the MMA's 128 rows:
// P costs 128 (K + V) multiplications a token, the carried state 2 K V.
// Why the products are cut between warps, how the output leaves, and the
// asynchronous first loads were each found by what the SM spent its time on:
// stores of rows from registers made the load-store unit the bound (TMA from
// shared memory instead), unrolled chunks the instruction cache (compact loops
// instead: issue slots 62 -> 48 % used), one issuing warp the queue of
// products.  The simplest form, one warp group doing each step in turn, took
// 664 and 531 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdio>
#include <string>

#include "../../include/fftconv.h"
#include "internal.h"
#include "tc_ptx.cuh"

namespace fftconv {
namespace {

using namespace tc;

constexpr int kChunk = 128;                   // tokens of a chunk: the rows of one MMA
constexpr int kStateWarps = 8;
constexpr uint32_t kWaitLimit = 1u << 16;      // polls of at most kPollNs: a wait gives up after about a second
constexpr uint32_t kPollNs = 20000;
constexpr int kMaxRoles = 3;

__device__ int g_status;                      // FFTCONV_ERR_TIMEOUT once a wait gave up

struct Role {
    int x, y, z;                              // tensor maps of the three sides
    int x_div, y_div, z_div;                  // heads of the call per head of the tensor
    int out_map;                              // tensor map of the output
    int rev;                                  // backward in time
    int out_f32;                              // fp32 partial sums of shared heads
    int kd, vd;                               // key and value dims
    int init_t;                               // init is stored [vd][kd]
    float a_in, a_carry, key_scale;
    void* out;
    int64_t out_b, out_t, out_h;
    const float* init;                        // [seq][H][kd][vd], or null: zeros
    float* fin;                               // carry behind the last token, or null
    float* seg;                               // states of cut sequences' segments [sid][H][vd][kd]: a lane's row, so that loads coalesce
};

struct Params {
    CUtensorMap maps[7];
    Role role[kMaxRoles];
    const float* log_decay;
    const int32_t* cu;
    int64_t T;
    int nroles, H, nseq, nper, seg_len, max_seg, max_cut, max_seqs;   // nper: segments of a sequence (unpacked)
    int in_place;                             // the final states take the initial states' place
    int4* table;                              // packed and cut: la_plan's segments, two words each
    int4* cuts;                               // ... those of sequences in two or more
    int4* seqs;                               // ... and these sequences: which, its first segment's sid, their number
};

// A segment: which sequence, which of its segments and tokens.
struct Segment {
    int seq, idx, count, n;                   // n: tokens
    int t0, b;                                // first token's coordinates
    int sid;                                  // place among the segments of cut sequences
};

// The segment that the order-th CTA of a head and role takes (seq = -1: none).
// Sequences without tokens have one empty segment.
__device__ Segment find_segment(const Params& p, const int4* table, int order) {
    if (table) {
        const int4 u = table[2 * (int64_t)order], v = table[2 * (int64_t)order + 1];
        return Segment{u.x, u.y, u.z, u.w, v.x, 0, v.y};
    }
    Segment s{order, 0, 1, (int)p.T, 0, 0, order};
    if (p.cu) {                                               // packed, not cut
        s.t0 = min(max(p.cu[order], 0), (int)p.T);
        s.n = min(max(p.cu[order + 1], s.t0), (int)p.T) - s.t0;
    } else {
        s.seq = s.b = order / p.nper;
        s.idx = order - s.seq * p.nper;
        s.count = p.nper;
        s.t0 = s.idx * p.seg_len;
        s.n = min(p.seg_len, (int)p.T - s.t0);
    }
    return s;
}

// sums of each of x over the threads before this one, and over the block
constexpr int kSums = 4;
struct Sums {
    int64_t v[kSums];
};
__device__ Sums sums_before(const Sums& x, Sums& all) {
    __shared__ Sums warps[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = (int)blockDim.x >> 5;
    Sums in = x, r;
    if (n == 1) {
        // (32 sequences of at most 2^22 segments: 32 bits)
#pragma unroll
        for (int i = 0; i < kSums; ++i) {
            int sum = (int)x.v[i];
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += y;
            }
            r.v[i] = sum - x.v[i];
            all.v[i] = __shfl_sync(0xffffffffu, sum, 31);
        }
        return r;
    }
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, in.v[i], d);
            if (lane >= d) in.v[i] += y;
        }
        r.v[i] = in.v[i] - x.v[i];
    }
    __syncthreads();                                          // (the last call's sums have been read)
    if (lane == 31) warps[warp] = in;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
        int64_t sum = 0;
        for (int w = 0; w < n; ++w) {
            if (w == warp) r.v[i] += sum;
            sum += warps[w].v[i];
        }
        all.v[i] = sum;
    }
    return r;
}

// Packed sequences that may be cut along time: the segments, those of over
// half the length first.  The CTAs run in about this order, and the short ones
// fill the SMs that are free early (8192 tokens in 9 sequences, 16 heads of
// 128/128: 112 us in the sequences' order, 102 in this one).  One block looks
// at all offsets, once: with each CTA looking for its own segment, 2048
// sequences of 64 tokens and 16 heads took 10.8 ms instead of 1.4.
// Only segments of sequences in two or more have states in the workspace, and
// a launch that sums them: a second list, in the same order, of at most
// 2 T / seg_len of them however many sequences there are; and the sequences
// themselves, whose order does not matter.  (Sums in 64 bits, and bounds:
// offsets that decrease can count more segments than there is room for.)
__global__ void __launch_bounds__(1024) la_plan(const __grid_constant__ Params p) {
    struct Look {
        int start, len, cnt;
        Sums n;                                               // segments over half the length, all; both of cut sequences
    };
    auto look = [&](int i) {
        Look s{0, 0, 0, {{0, 0, 0, 0}}};
        if (i >= p.nseq) return s;
        s.start = min(max(p.cu[i], 0), (int)p.T);
        s.len = min(max(p.cu[i + 1], s.start), (int)p.T) - s.start;
        s.cnt = max(1, (s.len + p.seg_len - 1) / p.seg_len);
        const int longs = s.cnt - (s.len - (s.cnt - 1) * p.seg_len <= p.seg_len / 2);
        s.n = Sums{{longs, s.cnt, s.cnt > 1 ? longs : 0, s.cnt > 1 ? s.cnt : 0}};
        return s;
    };
    __shared__ int nseqs;
    if (threadIdx.x == 0) nseqs = 0;
    __syncthreads();
    Sums total{{0, 0, 0, 0}}, all, before = total;
    const bool once = p.nseq <= (int)blockDim.x;              // (the one scan has the totals too)
    if (!once) {
        Sums mine = total;
        for (int i = threadIdx.x; i < p.nseq; i += blockDim.x) {
            const Look s = look(i);
            for (int e = 0; e < kSums; ++e) mine.v[e] += s.n.v[e];
        }
        sums_before(mine, total);
    }
    for (int base = 0; base < p.nseq; base += blockDim.x) {
        const int i = base + (int)threadIdx.x;
        const Look s = look(i);
        Sums at = sums_before(s.n, all);
        if (once) total = all;
        for (int e = 0; e < kSums; ++e) at.v[e] += before.v[e];
        const bool fits = at.v[1] + s.cnt <= p.max_seg && at.v[3] + s.n.v[3] <= p.max_cut;
        if (s.cnt > 1 && fits) {
            const int at_seq = atomicAdd(&nseqs, 1);
            if (at_seq < p.max_seqs) p.seqs[at_seq] = make_int4(i, (int)at.v[3], s.cnt, 0);
        }
        for (int j = 0; j < s.cnt; ++j) {
            const int4 u = make_int4(fits ? i : -1, j, s.cnt, min(p.seg_len, s.len - j * p.seg_len));
            const int4 v = make_int4(s.start + j * p.seg_len, s.cnt > 1 ? (int)at.v[3] + j : 0, 0, 0);
            auto list = [&](int4* table, int64_t most, int e) {
                const int64_t order = j < (int)s.n.v[0] ? at.v[e] + j : total.v[e] + at.v[e + 1] - at.v[e];
                if (order >= most) return false;
                table[2 * order] = u;
                table[2 * order + 1] = v;
                return true;
            };
            const bool room = list(p.table, p.max_seg, 0);
            if (!(s.cnt > 1 && list(p.cuts, p.max_cut, 2)) && !room) break;
        }
        for (int e = 0; e < kSums; ++e) before.v[e] += all.v[e];
    }
    const int4 none = make_int4(-1, 0, 0, 0);
    for (int64_t e = total.v[1] + threadIdx.x; e < p.max_seg; e += blockDim.x) p.table[2 * e] = none;
    for (int64_t e = total.v[3] + threadIdx.x; e < p.max_cut; e += blockDim.x) p.cuts[2 * e] = none;
    __syncthreads();
    for (int e = nseqs + (int)threadIdx.x; e < p.max_seqs; e += (int)blockDim.x) p.seqs[e] = none;
}

// g^n for g = exp(ld), the product ld * n carried in two fp32 parts.  Decays
// below exp(-1e4) are 0 from the first power on, like -inf.
__device__ __forceinline__ float decay_power(float ld, float n) {
    ld = ld < -1e4f ? -1e4f : ld;
    const float p = ld * n;
    const float e = expf(p);
    return n == 0.f ? 1.f : isinf(e) ? e : fmaf(e, fmaf(ld, n, -p), e);
}

// g^n in two fp32 parts, for powers that are applied again and again: a walk
// over 512 chunks with g^128 rounded once was off by 1.7e-5, in a direction.
// Decays of over a half keep one part: what they weigh is gone before the
// error counts (X factors of it: 2 X 2^-23 relative of exp(-X)).
__device__ __forceinline__ float2 decay_power2(float ld, float n) {
    const float p = ld * n;
    if (!(fabsf(p) < 0.5f)) return make_float2(decay_power(ld, n), 0.f);
    const float e = expm1f(p), d = fmaf(fmaf(ld, n, -p), 1.f + e, e), hi = 1.f + d;
    return make_float2(hi, (1.f - hi) + d);
}

__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a));
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t (&r)[32]) {
    tmem_st16(a, r);
    tmem_st16(a + 16, r + 16);
}

__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int d, int h, int t, int b,
                                         uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(d), "r"(h), "r"(t), "r"(b), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_store(const CUtensorMap* map, const void* src, int d, int h, int t, int b) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(map),
                 "r"(d), "r"(h), "r"(t), "r"(b), "r"(smem_u32(src))
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// until the issuing thread's stores have read their shared memory
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// Four 8 x 8 tiles of 16-bit values, each transposed: a lane gives the address
// of row lane % 8 of tile lane / 8 and receives column lane / 4, rows
// 2 (lane % 4) and + 1, of every tile.
__device__ __forceinline__ void ldmatrix4_trans(const void* row, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(row))
                 : "memory");
}
// 16 TMEM lanes x 16 columns: register 2 i + x holds lane 8 x + laneid / 4,
// column 4 i + laneid % 4.
__device__ __forceinline__ void tmem_st_16x16(uint32_t a, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// 16-bit arithmetic of the two types: packing with round to nearest even, and
// the two halves as fp32.
template <bool F16>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    if constexpr (F16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <bool F16>
__device__ __forceinline__ float2 unpack(uint32_t v) {
    if constexpr (F16) {
        __half2 h;
        *reinterpret_cast<uint32_t*>(&h) = v;
        return __half22float2(h);
    } else {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ void scale2(uint32_t& a, uint32_t& b, float2 f) {
    const float2 r = mul2(make_float2(__uint_as_float(a), __uint_as_float(b)), f);
    a = __float_as_uint(r.x);
    b = __float_as_uint(r.y);
}

template <bool F16>
__device__ __forceinline__ uint4 pack8(const uint32_t* s) {
    uint4 v;
    v.x = pack<F16>(__uint_as_float(s[0]), __uint_as_float(s[1]));
    v.y = pack<F16>(__uint_as_float(s[2]), __uint_as_float(s[3]));
    v.z = pack<F16>(__uint_as_float(s[4]), __uint_as_float(s[5]));
    v.w = pack<F16>(__uint_as_float(s[6]), __uint_as_float(s[7]));
    return v;
}

// 2^e with the largest exponent that keeps amax * 2^e below 2^15 (1 for 0,
// inf and NaN): the exact scale of an fp16 operand.
__device__ __forceinline__ float fp16_scale(float amax) {
    const int ex = (int)((__float_as_uint(amax) >> 23) & 255);
    if (ex == 0 || ex == 255) return 1.f;
    const int e = min(max(14 - (ex - 127), -60), 60);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Wait for the phase with the given parity, suspended rather than polling;
// false once *abort is set or the limit is reached.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, const volatile int* abort) {
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(kPollNs)
            : "memory");
        if (ok) return true;
        if (ld_shared_volatile(abort)) return false;
    }
    return false;
}

// Parts of the weighted keys and how they lie in TMEM.  EXACT: the state itself
// is a result, fp32, so all 24 bits of a weighted bf16 key count (three parts;
// fp16: two, 22 bits).  Else the state only goes into 16-bit outputs:
//   64 channels: one part, rounded, and the carry's copy in two parts;
//   128 channels (no room for a second copy): two parts, and the copy rounded.
// Either way a carried term is rounded once, like a term of P.
template <int KP, int VP, bool F16, bool STATE_ONLY, bool EXACT>
struct Layout {
    static constexpr bool Single = KP == 64 && !EXACT;
    // 64 channels, EXACT: two parts are stacked on the 128 rows of one MMA,
    // and the state is kept as the two rows' sum
    static constexpr bool Stacked = KP == 64 && EXACT;
    static constexpr int Parts = Single ? 1 : F16 || !EXACT ? 2 : 3;
    // state warps with rows of the state
    static constexpr int Live = Single ? 4 : kStateWarps;
    // beside P and the output three parts do not fit: the first one waits for
    // the others' columns
    static constexpr bool Late = !STATE_ONLY && Parts == 3;
    static constexpr int KtCols = Stacked ? (Parts == 3 && !Late ? 128 : 64) : Late ? 128 : Parts * 64;   // (Single: 64)
    // where the columns suffice, a chunk's keys are weighed while the last one's are multiplied
    static constexpr int KtBufs = STATE_ONLY || (KP == 64 && VP == 128 && !Late) ? 2 : 1;
    // the carry product has columns of its own (else P z is added to it, once it is weighted)
    static constexpr bool SplitOut = KP == 64 && VP == 64;
    // groups of row warps, which take chunks in turn, each with a score tile
    static constexpr int Groups = VP == 64 ? 2 : 1;
    static constexpr int RowWarps = 4 * Groups;
    static constexpr int LoadWarp = RowWarps + kStateWarps, MmaWarp = LoadWarp + 1, StateMmaWarp = LoadWarp + 2,
                         ScoreWarp = LoadWarp + 3;
    static constexpr int Threads = (RowWarps + kStateWarps + 4) * 32;
    static constexpr int XBytes = KP * kChunk * 2, ZBytes = VP * kChunk * 2;
    static constexpr int OffY = STATE_ONLY ? 0 : XBytes, OffZ = OffY + XBytes, StageBytes = OffZ + ZBytes;
    static constexpr int CarryBytes = STATE_ONLY && !Stacked ? 0 : 128 * VP * 2;   // 64 channels: two copies
    static constexpr int Stages = StageBytes <= 49152 ? 4 : StageBytes <= 65536 ? 3 : 2;
    static constexpr int OffCarry = Stages * StageBytes;
    static constexpr int OffTab = OffCarry + CarryBytes;      // a g^|d| or 0, d = j - i in [-32, 31]
    static constexpr int OffCol = OffTab + 64 * 4;            // column weights of an unmasked block of P
    static constexpr int OffPow = OffCol + 32 * 4;            // g^e, e <= 128; g^128 in two parts (129, 130)
    static constexpr int OffKw = OffPow + 132 * 4;            // key weights of the chunk
    static constexpr int OffMisc = OffKw + 128 * 4;           // abort (word 6), TMEM base (7), scales
    static constexpr int OffBar = OffMisc + 128;
    static constexpr int Bars = 29 + (F16 ? 4 : 0);
    static constexpr int OffMax = OffBar + (Bars + 1) / 2 * 16;   // (fp16) channel maxima [2][state warps][32]
    static constexpr int Bytes = OffMax + (F16 ? 2 * kStateWarps * 32 * 2 : 0);
    // TMEM columns
    static constexpr int S = 0, O = S + Groups * 128, Oc = SplitOut ? O + VP : O, C = STATE_ONLY ? 0 : Oc + VP,
                         Kt = C + VP;
    static_assert(Bytes <= 232448, "shared memory");
    static_assert(Kt + KtBufs * KtCols <= 512, "TMEM columns");
};

// One CTA: one (segment, head, role).  Row warps (one or two groups of four
// that take chunks in turn) own the token rows: P and the output, which
// leaves through the query tile's shared memory.  Eight state warps keep the
// state in registers (its decay, its 16-bit copy for the next product) and
// weigh the keys, transposed into TMEM.  One warp issues the loads, three the
// MMAs (scores; carry product and P z; the chunk's own state), so that none
// waits behind another's operands.  Only the carry product waits for the
// state, so chunks overlap.
//
// Rounding: P, and the weighted keys or the carry's copy (Layout), are rounded
// once to the 16-bit type: their products are the two halves of the output,
// each with the error of one rounding of it.  FINE: P in two parts, 16 bits or
// more, for calls of few tokens (kFineTokens), and so the copy of the state in
// front of a sequence that is one chunk.  fp16 operands are scaled by
// exact powers of two (P by row, the carry's copy by its largest value, the
// weighted keys by channel), so that nothing overflows fp16's range or falls
// below it.
template <int KP, int VP, bool F16, bool STATE_ONLY, bool EXACT, bool FINE>
__global__ void __launch_bounds__(Layout<KP, VP, F16, STATE_ONLY, EXACT>::Threads, 1)
    la_kernel(const __grid_constant__ Params p) {
    using L = Layout<KP, VP, F16, STATE_ONLY, EXACT>;
    constexpr bool kAhead = L::KtBufs == 2;                   // keys weighed one chunk ahead (never Late)
    constexpr int NA = L::Groups;
    extern __shared__ __align__(1024) uint8_t smem[];
    float* tab = reinterpret_cast<float*>(smem + L::OffTab);
    float* colw = reinterpret_cast<float*>(smem + L::OffCol);
    float* pw = reinterpret_cast<float*>(smem + L::OffPow);
    float* kw = reinterpret_cast<float*>(smem + L::OffKw);
    volatile int* misc = reinterpret_cast<volatile int*>(smem + L::OffMisc);
    volatile int* abort_flag = misc + 6;
    uint32_t* tmem_sh = reinterpret_cast<uint32_t*>(smem + L::OffMisc) + 7;
    volatile float* carry_inv = reinterpret_cast<volatile float*>(misc + 8);      // [4] by chunk
    volatile float* amax_sh = reinterpret_cast<volatile float*>(misc + 12);       // [2][8]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OffBar);
    uint64_t* full = bars;                                    // [Stages] loads
    uint64_t* empty = bars + 4;                               // [Stages] MMAs and output are done with a stage
    uint64_t* bar_s = bars + 8;                               // [Groups] scores
    uint64_t* bar_o = bars + 10;                              // [Groups] carry product
    uint64_t* bar_pv = bars + 12;                             // [Groups] output
    uint64_t* p_ready = bars + 14;                            // [Groups] P written, carry product weighted
    uint64_t* o_free = bars + 16;                             // [Groups] output read
    uint64_t* bar_st = bars + 18;                             // the chunk's own state
    uint64_t* bar_kt = bars + 19;                             // its first parts (Late only)
    uint64_t* late_ready = bars + 21;
    uint64_t* carry_ready = bars + 22;
    uint64_t* z_ready = bars + 23;                            // rows behind a packed sequence zeroed
    uint64_t* wgb_bar = bars + 24;
    uint64_t* c_free = bars + 25;                             // the chunk's own state read
    uint64_t* bar_fin = bars + 26;                            // all MMA warps
    // keys weighed, a barrier for each of their buffers: with two of them the
    // state warps may be done with chunk c + 1 before the MMA warp has seen
    // chunk c, and two phases of one barrier look like none
    auto kt_ready = [&](int c) { return c % L::KtBufs ? bars + 27 : bars + 20; };
    uint64_t* pow_ready = bars + 28;                          // g^128's two parts
    uint64_t* pair_bar = bars + 29;                           // [4] (fp16) the two state warps of the same channels

    const int tid = threadIdx.x;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int lane = tid & 31;
    const int role_i = blockIdx.x % p.nroles;
    const int h = (blockIdx.x / p.nroles) % p.H;
    const int order = blockIdx.x / (p.nroles * p.H);
    const Role& r = p.role[role_i];
    const bool rev = r.rev != 0;

    // a segment's chunks, and whether it is the first or last in the role's
    // direction of time; a cut sequence's last own state only matters where the
    // final state is a result
    auto first_of = [&](int idx, int count) { return rev ? idx == count - 1 : idx == 0; };
    auto chunks_of = [&](const Segment& s) {
        if (s.seq < 0 || (STATE_ONLY && first_of(s.count - 1 - s.idx, s.count) && (s.count == 1 || r.fin == nullptr)))
            return 0;
        return (s.n + kChunk - 1) / kChunk;
    };
    auto load_chunk = [&](int c, int nch, int t0, int b) {    // by one thread
        const int st = c % L::Stages, t = t0 + (rev != STATE_ONLY ? nch - 1 - c : c) * kChunk;
        const int hx = h / r.x_div, hy = h / r.y_div, hz = h / r.z_div;
        uint8_t* base = smem + st * L::StageBytes;
        mbar_expect_tx(&full[st], L::StageBytes);
        for (int d = 0; d < KP; d += 64) tma_load(base + L::OffY + d * 256, &p.maps[r.y], d, hy, t, b, &full[st]);
        if (!STATE_ONLY)
            for (int d = 0; d < KP; d += 64) tma_load(base + d * 256, &p.maps[r.x], d, hx, t, b, &full[st]);
        for (int d = 0; d < VP; d += 64) tma_load(base + L::OffZ + d * 256, &p.maps[r.z], d, hz, t, b, &full[st]);
    };

    // (without tokens, and without a state to pass on, the whole CTA leaves)
    const Segment s = find_segment(p, STATE_ONLY ? p.cuts : p.table, order);
    if (chunks_of(s) == 0 && (STATE_ONLY || s.seq < 0 || r.fin == nullptr)) return;
    if (warp == L::LoadWarp) {
        if (lane == 0) {
            for (int i = 0; i < 4; ++i) {
                mbar_init(&full[i], 1);
                mbar_init(&empty[i], STATE_ONLY ? 1 : 6);     // two MMA warps, four row warps
            }
            for (int i = 8; i < 14; ++i) mbar_init(bars + i, 1);
            for (int i = 14; i < 18; ++i) mbar_init(bars + i, 4);
            mbar_init(bar_st, 1);
            mbar_init(pow_ready, 1);
            mbar_init(bar_kt, 1);
            for (int i = 20; i < 26; ++i) mbar_init(bars + i, L::Live);
            mbar_init(bar_fin, STATE_ONLY ? 1 : 3);
            mbar_init(bars + 27, L::Live);
            if constexpr (F16)
                for (int i = 0; i < 4; ++i) mbar_init(&pair_bar[i], 2);
            *abort_flag = 0;
            fence_barrier_init();
            fence_proxy_async_smem();                         // the loads' engine sees the barriers
            // the first loads go out while the other warps set up
            const int nch = chunks_of(s);
            for (int c = 0; c < min(nch, L::Stages); ++c) load_chunk(c, nch, s.t0, s.b);
        }
    } else if (warp == L::MmaWarp) {
        tmem_alloc(tmem_sh, 512);
        tmem_relinquish();
    } else if (warp >= L::RowWarps && warp < L::RowWarps + 4) {
        const float ld = p.log_decay[h];
        const int i = tid - L::RowWarps * 32;
        const float w = decay_power(ld, (float)i);
        pw[i] = w;
        if (i == 127) pw[128] = decay_power(ld, 128.f);
        if (i < 32) {
            tab[32 + (rev ? i : -i)] = r.a_in * w;
            if (i) tab[32 - (rev ? i : -i)] = 0.f;
            colw[rev ? i : 31 - i] = r.a_in * w;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = __shfl_sync(0xffffffffu, *tmem_sh, 0);
    const int seq = s.seq, n = s.n, t0 = s.t0, b = s.b;
    const bool first = first_of(s.idx, s.count);
    const int nch = chunks_of(s);
    const bool has_init = !STATE_ONLY && (first ? r.init != nullptr : true);
    const bool want_fin = STATE_ONLY || (s.count == 1 && r.fin != nullptr);
    // one chunk: the copy of its initial state has a second part, in the next
    // stage's place (128 channels) or that of the second sums, which are zero
    const bool copy_in_two = L::Single || (FINE && nch == 1);

    auto wait = [&](uint64_t* bar, uint32_t phase) -> bool {
        return __all_sync(0xffffffffu, wait_phase(bar, phase & 1, abort_flag));
    };
    auto fail = [&]() {
        *abort_flag = 1;
        atomicExch(&g_status, FFTCONV_ERR_TIMEOUT);
    };
    auto arrive = [&](uint64_t* bar) {                        // one arrival a warp
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    // chunk c of the role's direction: its first token and number of tokens.
    // (A segment's own state is summed from its end, so that what the next
    // launch reads first is what this one leaves in L2.)
    auto chunk_at = [&](int c) { return (rev != STATE_ONLY ? nch - 1 - c : c) * kChunk; };
    auto chunk_n = [&](int c) { return min(kChunk, n - chunk_at(c)); };
    constexpr uint32_t kFmt = F16 ? 0u : (1u << 7) | (1u << 10);
    constexpr uint32_t kTransB = 1u << 16;
    // ks products of 16 tokens: A in TMEM, B the value tile
    auto token_mma = [&](uint32_t d, uint32_t a, uint64_t d_z, uint32_t id, int ks, uint32_t acc) {
        if (ks == 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) mma_ts_warp(d, a + k * 8, d_z + (uint64_t)(k * 128), id, k > 0 ? 1u : acc);
        } else {
            for (int k = 0; k < ks; ++k) mma_ts_warp(d, a + k * 8, d_z + (uint64_t)(k * 128), id, k > 0 ? 1u : acc);
        }
    };

    // ... and with A = P, each 32 columns' two parts side by side
    auto row_mma = [&](uint32_t d, uint32_t a, uint64_t d_z, uint32_t id, int ks, uint32_t acc) {
        auto step = [&](int k) {
            mma_ts_warp(d, a + (k >> 1) * 32 + (k & 1) * 8, d_z + (uint64_t)(k * 128), id, k > 0 ? 1u : acc);
        };
        if (ks == 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) step(k);
        } else {
            for (int k = 0; k < ks; ++k) step(k);
        }
    };

    if (warp == L::LoadWarp) {
        // ------------------------------------------------------- loads ---
        if (lane == 0) {
            int issued = min(nch, L::Stages);
            for (int c = L::Stages; c < nch; ++c) {
                if (!wait_phase(&empty[c % L::Stages], ((c / L::Stages) - 1) & 1, abort_flag)) {
                    fail();
                    break;
                }
                load_chunk(c, nch, t0, b);
                issued = c + 1;
            }
            // nothing of this CTA's loads is in flight when it ends
            for (int c = max(0, issued - L::Stages); c < issued; ++c)
                for (uint32_t i = 0; i < kWaitLimit; ++i)
                    if (mbar_try_wait(&full[c % L::Stages], (c / L::Stages) & 1)) break;
        }
    } else if (warp == L::MmaWarp) {
        // ------------------------------------------- MMAs of the rows ---
        if constexpr (!STATE_ONLY) {
            const uint32_t id_z = idesc_f16_f32(128, VP) | kFmt | kTransB;
            const uint32_t sb = smem_u32(smem), t_o = tbase + L::O, t_oc = tbase + L::Oc;
            const uint64_t d_carry = make_desc(sb + L::OffCarry, 128 * 128, 1024, 2);
            bool ok = true;
            for (int c = 0; c < nch; ++c) {
                const int st = c % L::Stages, ga = c % NA;
                const int ks = (chunk_n(c) + 15) / 16;
                const bool carry = c > 0 || has_init;
                const uint32_t base = sb + st * L::StageBytes;
                const uint64_t d_x = make_desc(base, 16, 1024, 2);
                const uint64_t d_z = make_desc(base + L::OffZ, 16384, 1024, 2);
                ok = wait(&full[st], c / L::Stages) && wait(carry_ready, c) &&
                     (c == 0 || wait(&o_free[(c - 1) % NA], (c - 1) / NA));
                if (!ok) break;
                tc_fence_after();
                if (carry) {
                    // (64 channels: the query's four steps against both halves of the state)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int kx = k % (KP / 16);
                        const uint64_t step = (uint64_t)((kx >> 2) * 16384 + (kx & 3) * 32) >> 4;
                        mma_ss_warp(t_oc, d_x + step, d_carry + (uint64_t)(k * 128), id_z, k > 0);
                    }
                    if constexpr (FINE && KP == 128) {
                        if (copy_in_two) {
                            const uint64_t d_rest = make_desc(sb + L::StageBytes, 128 * 128, 1024, 2);
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const uint64_t step = (uint64_t)((k >> 2) * 16384 + (k & 3) * 32) >> 4;
                                mma_ss_warp(t_oc, d_x + step, d_rest + (uint64_t)(k * 128), id_z, 1u);
                            }
                        }
                    }
                }
                tc_commit_warp(&bar_o[ga]);
                ok = wait(&p_ready[ga], c / NA);
                if (ok && p.cu && chunk_n(c) < kChunk) ok = wait(z_ready, 0);
                if (!ok) break;
                tc_fence_after();
                const uint32_t t_p = tbase + L::S + ga * 128;
                const uint32_t acc = carry && !L::SplitOut ? 1u : 0u;
                if constexpr (FINE) row_mma(t_o, t_p + 16, d_z, id_z, ks, acc);
                row_mma(t_o, t_p, d_z, id_z, ks, FINE ? 1u : acc);
                tc_commit_warp(&bar_pv[ga]);
                tc_commit_warp(&empty[st]);
            }
            if (!ok) fail();
            tc_commit_warp(bar_fin);
        }
    } else if (warp == L::ScoreWarp) {
        // ----------------------------------------- MMAs of the scores ---
        if constexpr (!STATE_ONLY) {
            const uint32_t id_s = idesc_f16_f32(128, 128) | kFmt;
            const uint32_t sb = smem_u32(smem);
            bool ok = true;
            for (int c = 0; c < nch; ++c) {
                const int st = c % L::Stages, ga = c % NA;
                const uint32_t base = sb + st * L::StageBytes;
                const uint64_t d_x = make_desc(base, 16, 1024, 2), d_y = make_desc(base + L::OffY, 16, 1024, 2);
                // the loads are there, and the score tile's last P is used up
                ok = wait(&full[st], c / L::Stages) && (c < NA || wait(&bar_pv[ga], c / NA - 1));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < KP / 16; ++k) {
                    const uint64_t step = (uint64_t)((k >> 2) * 16384 + (k & 3) * 32) >> 4;
                    mma_ss_warp(tbase + L::S + ga * 128, d_x + step, d_y + step, id_s, k > 0);
                }
                tc_commit_warp(&bar_s[ga]);
            }
            if (!ok) fail();
            tc_commit_warp(bar_fin);
        }
    } else if (warp == L::StateMmaWarp) {
        // ------------------------------ MMAs of the chunks' own states ---
        // The smallest parts first: the MMA truncates each sum, so few steps
        // should meet a large one.
        const uint32_t id = idesc_f16_f32(128, VP) | kFmt | kTransB;
        const uint32_t sb = smem_u32(smem), t_c = tbase + L::C;
        if (!STATE_ONLY && lane == 0) {
            // (by a warp that has nothing to do before the first keys are weighed)
            const float2 whole = decay_power2(p.log_decay[h], 128.f);
            pw[129] = whole.x;
            pw[130] = whole.y;
            mbar_arrive(pow_ready);
        }
        __syncwarp();
        bool ok = true;
        for (int c = 0; c < nch; ++c) {
            const int st = c % L::Stages;
            const int ks = (chunk_n(c) + 15) / 16;
            const uint64_t d_z = make_desc(sb + st * L::StageBytes + L::OffZ, 16384, 1024, 2);
            const uint32_t t_kt = tbase + L::Kt + c % L::KtBufs * L::KtCols;
            ok = wait(kt_ready(c), c / L::KtBufs);
            if (!ok) break;
            if (c + 1 < nch || want_fin) {
                if (kAhead && c > 0) ok = wait(c_free, c - 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int part = L::KtCols / 64 - 1; part >= 0; --part)
                    token_mma(t_c, t_kt + part * 64, d_z, id, ks, part == L::KtCols / 64 - 1 ? 0u : 1u);
                if constexpr (L::Late) {
                    tc_commit_warp(bar_kt);
                    ok = wait(late_ready, c);
                    if (!ok) break;
                    tc_fence_after();
                    token_mma(t_c, t_kt, d_z, id, ks, 1u);
                }
                tc_commit_warp(bar_st);
            }
            tc_commit_warp(&empty[st]);
        }
        if (!ok) fail();
        tc_commit_warp(bar_fin);
        // no MMA of any warp is in flight when TMEM is freed (also after a failed wait)
        for (uint32_t i = 0; i < kWaitLimit; ++i)
            if (__all_sync(0xffffffffu, mbar_try_wait(bar_fin, 0))) break;
    } else if (warp < L::RowWarps) {
        // -------------------------------------------------- token rows ---
        if constexpr (!STATE_ONLY) {
            const int ga = warp >> 2, wr = warp & 3;
            const int i = wr * 32 + lane;
            const uint32_t row = (uint32_t)(wr * 32) << 16;
            const uint32_t t_s = tbase + row + L::S + ga * 128;
            // a chunk's stage may be loaded again once its output's stores have
            // read it; with four stages that can wait until the next chunk's turn
            constexpr bool kDefer = L::Stages == 4;
            auto release = [&](int c) {
                if (lane == 0) {
                    bulk_wait_read();
                    mbar_arrive(&empty[c % L::Stages]);
                }
                __syncwarp();
            };
            for (int c = ga; c < nch; c += NA) {
                const int nv = chunk_n(c);
                const bool carry = c > 0 || has_init;
                const int jlo = rev ? i : 0, jhi = rev ? nv - 1 : i;
                const uint32_t t_o = tbase + row + L::O;
                // columns 32 blk .. 32 blk + 31 have nothing for this warp's rows
                auto masked = [&](int blk) { return (rev ? blk < wr : blk > wr) || blk * 32 >= nv; };
                auto weigh = [&](uint32_t (&s)[32], int blk, float scale) {
                    if (blk != wr) {
                        // g^|i-j| as (row to the block's near edge) x (edge to
                        // column): both at most 1, four columns a load
                        const float f = pw[rev ? blk * 32 - i : i - blk * 32 - 31] * scale;
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 w = *reinterpret_cast<const float4*>(colw + j);
                            scale2(s[j], s[j + 1], mul2(make_float2(f, f), make_float2(w.x, w.y)));
                            scale2(s[j + 2], s[j + 3], mul2(make_float2(f, f), make_float2(w.z, w.w)));
                        }
                    } else {
                        // on the diagonal: the table is zero beyond it
                        const float* w = tab + 32 - lane;
#pragma unroll
                        for (int j = 0; j < 32; j += 2)
                            scale2(s[j], s[j + 1], F16 ? mul2(make_float2(w[j], w[j + 1]), make_float2(scale, scale))
                                                       : make_float2(w[j], w[j + 1]));
                    }
                    if (nv < kChunk) {
                        // columns behind the end may be another sequence's inf or NaN
#pragma unroll
                        for (int j = 0; j < 32; ++j) s[j] = blk * 32 + j >= jlo && blk * 32 + j <= jhi ? s[j] : 0u;
                    }
                };
                if (!wait(&bar_s[ga], c / NA)) { fail(); break; }
                tc_fence_after();
                if (kDefer && c >= NA) release(c - NA);
                float scale = 1.f;
                if constexpr (F16) {
                    float amax = 0.f;
#pragma unroll 1
                    for (int blk = 0; blk < 4; ++blk) {
                        if (masked(blk)) continue;
                        uint32_t s[32];
                        tmem_ld32(t_s + blk * 32, s);
                        tc_wait_ld();
                        // (the weights are at most a, or where g is above 1 a
                        // times the power for the row's farthest column; a
                        // score far above the weighted ones costs nothing
                        // within 2^28)
                        if (nv == kChunk) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) amax = fmaxf(amax, fabsf(__uint_as_float(s[j])));
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (blk * 32 + j >= jlo && blk * 32 + j <= jhi)
                                    amax = fmaxf(amax, fabsf(__uint_as_float(s[j])));
                        }
                    }
                    const int far = max(0, jhi - jlo), half = far / 2;    // (in two steps: the power itself may overflow)
                    scale = fp16_scale(amax * fmaxf(fabsf(r.a_in), fabsf(r.a_in) * pw[half] * pw[far - half]));
                }
                // P (16 bit) lies over the score columns that this thread has
                // read: each 32 columns' words, and behind them what they leave out
#pragma unroll 1
                for (int blk = 0; blk < 4; ++blk) {
                    uint32_t s[32], pk[16];
                    if (masked(blk)) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) pk[j] = 0u;
                        if constexpr (FINE) tmem_st16(t_s + blk * 32 + 16, pk);
                    } else {
                        tmem_ld32(t_s + blk * 32, s);
                        tc_wait_ld();
                        weigh(s, blk, scale);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            pk[j] = pack<F16>(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
                        if constexpr (FINE) {
                            uint32_t lo[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float2 hi = unpack<F16>(pk[j]);
                                lo[j] = pack<F16>(__uint_as_float(s[2 * j]) - hi.x, __uint_as_float(s[2 * j + 1]) - hi.y);
                            }
                            tmem_st16(t_s + blk * 32 + 16, lo);
                        }
                    }
                    tmem_st16(t_s + blk * 32, pk);
                }
                const float inv = F16 ? 1.f / scale : 1.f;
                float f = r.a_carry * pw[min(128, max(0, rev ? nv - 1 - i : i + 1))];
                if constexpr (L::SplitOut) {
                    tc_wait_st();
                    tc_fence_before();
                    arrive(&p_ready[ga]);
                }
                if (!wait(&bar_o[ga], c / NA)) { fail(); break; }
                tc_fence_after();
                if constexpr (F16) {
                    if (carry) f *= carry_inv[c & 3];
                }
                if (carry && !L::SplitOut) {
                    f *= scale;
#pragma unroll 1
                    for (int blk = 0; blk < VP / 32; ++blk) {
                        uint32_t s[32];
                        tmem_ld32(t_o + blk * 32, s);
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; j += 2) scale2(s[j], s[j + 1], make_float2(f, f));
                        tmem_st32(t_o + blk * 32, s);
                    }
                }
                if constexpr (!L::SplitOut) {
                    tc_wait_st();
                    tc_fence_before();
                    arrive(&p_ready[ga]);
                }
                if (!wait(&bar_pv[ga], c / NA)) { fail(); break; }
                tc_fence_after();
                const int st = c % L::Stages, t = t0 + chunk_at(c);
                // Through the query tile, which no MMA reads any more: each
                // warp stages its 32 rows in 4 KB pieces (rows of 128 bytes,
                // 128-byte swizzle) and stores them by TMA, which leaves out
                // what lies outside the tensor.  The last rows of a packed
                // sequence, which others follow, are stored directly.
                const bool direct = p.cu && nv < kChunk;
                constexpr int kSlots = KP / 64;
                uint8_t* slot0 = smem + st * L::StageBytes + wr * 4096;
                int piece = 0;
                auto send = [&](int d0) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store(&p.maps[r.out_map], slot0 + piece % kSlots * 16384, d0, h, t + wr * 32, b);
                        bulk_commit();
                    }
                    ++piece;
                };
                auto reuse = [&]() {                          // a piece's place, once its store has read it
                    if (piece >= kSlots) {
                        if (lane == 0) bulk_wait_read();
                        __syncwarp();
                    }
                };
#pragma unroll 1
                for (int blk = 0; blk < VP / 32; ++blk) {
                    uint32_t s[32];
                    tmem_ld32(t_o + blk * 32, s);
                    if constexpr (L::SplitOut) {
                        uint32_t x[32];
                        if (carry) tmem_ld32(t_o + VP + blk * 32, x);
                        tc_wait_ld();
                        if constexpr (F16) {
#pragma unroll
                            for (int j = 0; j < 32; j += 2) scale2(s[j], s[j + 1], make_float2(inv, inv));
                        }
                        if (carry) {
#pragma unroll
                            for (int j = 0; j < 32; j += 2) {
                                const float2 y = fma2(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])),
                                                      make_float2(f, f),
                                                      make_float2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])));
                                s[j] = __float_as_uint(y.x);
                                s[j + 1] = __float_as_uint(y.y);
                            }
                        }
                    } else {
                        tc_wait_ld();
                        if constexpr (F16) {
#pragma unroll
                            for (int j = 0; j < 32; j += 2) scale2(s[j], s[j + 1], make_float2(inv, inv));
                        }
                    }
                    if (blk == VP / 32 - 1) {
                        tc_fence_before();
                        arrive(&o_free[ga]);
                    }
                    if (direct) {
                        const int64_t at = (int64_t)b * r.out_b + (int64_t)(t + i) * r.out_t + (int64_t)h * r.out_h;
                        if (i < nv && r.out_f32) {
                            float* o = reinterpret_cast<float*>(r.out) + at + blk * 32;
#pragma unroll
                            for (int j = 0; j < 32; j += 4)
                                if (blk * 32 + j < r.vd)
                                    *reinterpret_cast<uint4*>(o + j) = make_uint4(s[j], s[j + 1], s[j + 2], s[j + 3]);
                        } else if (i < nv) {
                            uint16_t* o = reinterpret_cast<uint16_t*>(r.out) + at + blk * 32;
#pragma unroll
                            for (int j = 0; j < 32; j += 8)
                                if (blk * 32 + j < r.vd) *reinterpret_cast<uint4*>(o + j) = pack8<F16>(s + j);
                        }
                        __syncwarp();
                    } else if (r.out_f32) {
                        reuse();
                        uint8_t* dst = slot0 + piece % kSlots * 16384 + lane * 128;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<uint4*>(dst + ((j ^ (lane & 7)) << 4)) =
                                make_uint4(s[4 * j], s[4 * j + 1], s[4 * j + 2], s[4 * j + 3]);
                        send(blk * 32);
                    } else {
                        if (!(blk & 1)) reuse();
                        uint8_t* dst = slot0 + piece % kSlots * 16384 + lane * 128;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<uint4*>(dst + ((((blk & 1) * 4 + j) ^ (lane & 7)) << 4)) =
                                pack8<F16>(s + 8 * j);
                        if (blk & 1) send(blk * 32 - 32);
                    }
                }
                if (!kDefer) release(c);
            }
            if (lane == 0) bulk_wait_read();                  // (also after a failed wait)
        }
    } else {
        // -------------------------------------------------- state rows ---
        // Two warps share 32 rows of the MMA: each keeps half of the columns
        // and weighs half of the tokens.  64 channels: one half of the rows
        // carries the sums of the first (and third) part, the other those of
        // the second, or none (Single; its warps have nothing to do).  The
        // half with less work is on the schedulers whose row warps have more
        // columns: the last two forward in time, the first two backward.
        constexpr int kCols = VP / 2;
        const int sw = warp - L::RowWarps, bw = sw & 3, half = sw >> 2;
        const int d = bw * 32 + lane;
        const int ch = KP == 64 ? d & 63 : d;                 // key channel
        const bool heavy = KP == 128 || bw < 2 != rev;        // (warp-uniform)
        const bool second = L::Stacked && heavy;
        const int ts = L::Single ? half * 64 + ch : tid - L::RowWarps * 32;       // index among the live threads
        const int col0 = half * kCols;
        const uint32_t row = (uint32_t)(bw * 32) << 16;
        const int64_t mat = (int64_t)r.kd * r.vd;
        const int64_t at_seq = ((int64_t)seq * p.H + h) * mat, at_seg = ((int64_t)s.sid * p.H + h) * mat;
        // (fp16) powers of two on this channel's weighted keys: the chunk's at
        // hand, and the one's whose own state is read next
        float rs = 1.f, rs_done = 1.f;
        uint32_t sync_phase = 0;
        auto sync_b = [&]() -> bool {                         // bounded barrier of the state warps
            arrive(wgb_bar);
            return wait(wgb_bar, sync_phase++);
        };
        float state[kCols];
#pragma unroll
        for (int j = 0; j < kCols; ++j) state[j] = 0.f;
        // the state in front of the first chunk
        auto initial = [&]() {
            if (second || ch >= r.kd || (first && !r.init)) return;
            // (in place, a cut sequence's final state is already where the initial one was)
            const bool from_seg = !first || (p.in_place && s.count > 1);
            if (from_seg || r.init_t) {
                const float* src = (from_seg ? r.seg + at_seg : r.init + at_seq) + ch;
#pragma unroll
                for (int j = 0; j < kCols; ++j)
                    if (col0 + j < r.vd) state[j] = src[(int64_t)(col0 + j) * r.kd];
            } else {
                const float* src = r.init + at_seq + (int64_t)ch * r.vd + col0;
#pragma unroll
                for (int j = 0; j < kCols; j += 4)
                    if (col0 + j < r.vd) {
                        const float4 v = *reinterpret_cast<const float4*>(src + j);
                        state[j] = v.x;
                        state[j + 1] = v.y;
                        state[j + 2] = v.z;
                        state[j + 3] = v.w;
                    }
            }
        };
        const bool live = !L::Single || heavy;
        if (has_init && nch > 0 && live) initial();
        if (L::Stacked && L::KtCols == 128 && second) {
            // the third part has no second half
            const uint32_t zero[16] = {};
            for (int buf = 0; buf < L::KtBufs; ++buf) {
                tmem_st16(tbase + row + L::Kt + buf * L::KtCols + 64 + half * 32, zero);
                tmem_st16(tbase + row + L::Kt + buf * L::KtCols + 64 + half * 32 + 16, zero);
            }
        }
        // state <- g^n state + (own state of chunk c), once its products are
        // done; from the end: state <- state + g^(tokens after it) (own state).
        // What rounding a chunk's g^128 leaves out (drift) is put into the next
        // one's, so the product of any of them is off by one rounding or two.
        int behind = 0;
        float drift = 0.f, keep128 = 1.f;
        const float ld = STATE_ONLY ? p.log_decay[h] : 0.f;
        auto advance = [&](int c) -> bool {
            float after = 1.f;
            if constexpr (STATE_ONLY) {
                after = decay_power(ld, (float)behind);
                behind += chunk_n(c);
            } else if (c == 0) {
                if (!wait(pow_ready, 0)) return false;
                keep128 = pw[129];
                drift = -pw[130];
            }
            if (!wait(bar_st, c)) return false;
            tc_fence_after();
            const float keep = STATE_ONLY ? 1.f : chunk_n(c) == kChunk ? keep128 : pw[chunk_n(c)], inv = 1.f / rs_done;
#pragma unroll
            for (int blk = 0; blk < kCols / 32; ++blk) {
                uint32_t s[32];
                tmem_ld32(tbase + row + L::C + col0 + blk * 32, s);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float own = F16 ? __uint_as_float(s[j]) * inv : __uint_as_float(s[j]);
                    if constexpr (STATE_ONLY)
                        state[blk * 32 + j] = fmaf(after, own, state[blk * 32 + j]);
                    else
                        state[blk * 32 + j] = fmaf(keep, state[blk * 32 + j], own);
                }
            }
            if constexpr (!STATE_ONLY) {
                const float rest = pw[130] - drift;
                keep128 = pw[129] + rest;
                drift = (keep128 - pw[129]) - rest;
            }
            return true;
        };
        // the state in front of chunk c, and its copy for the carry product
        auto carry_on = [&](int c) -> bool {
            const bool carry = c > 0 || has_init;
            if (c > 0) {
                if (!advance(c - 1)) return false;
                if (kAhead) {
                    tc_fence_before();
                    arrive(c_free);
                }
            }
            if constexpr (!STATE_ONLY) {
                if (carry) {
                    float cs = 1.f;
                    if constexpr (F16) {
                        // common scale of the carry's 16-bit copy, from its largest value
                        float amax = 0.f;
#pragma unroll
                        for (int j = 0; j < kCols; ++j) amax = fmaxf(amax, fabsf(state[j]));
                        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
                        const int lw = L::Single ? half * 2 + (bw & 1) : sw;
                        if (lane == 0) amax_sh[(c & 1) * 8 + lw] = __uint_as_float(top);
                        if (!sync_b()) return false;
#pragma unroll
                        for (int w = 0; w < L::Live; ++w) amax = fmaxf(amax, amax_sh[(c & 1) * 8 + w]);
                        cs = fp16_scale(amax);
                    }
                    // the last carry product has read the copy
                    if (c > 0 && !wait(&bar_o[(c - 1) % NA], (c - 1) / NA)) return false;
                    if (F16 && ts == 0) carry_inv[c & 3] = 1.f / cs;
                    uint8_t* dst = smem + L::OffCarry + (L::Single ? ch : d) * 128;
                    const int rest_at = KP == 128 ? L::StageBytes - L::OffCarry : L::Single || d < 64 ? 64 * 128 : -64 * 128;
                    const bool no_copy = L::Stacked && copy_in_two && second;
#pragma unroll
                    for (int q = 0; q < kCols / 8; ++q) {
                        if (no_copy) break;
                        const int vc = col0 / 8 + q;
                        uint8_t* to = dst + (vc >> 3) * 16384 + (((vc & 7) ^ (d & 7)) << 4);
                        uint32_t v[4], rest[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float2 f = make_float2(state[q * 8 + 2 * e], state[q * 8 + 2 * e + 1]);
                            if constexpr (F16) f = mul2(f, make_float2(cs, cs));
                            v[e] = pack<F16>(f.x, f.y);
                            if (copy_in_two) {
                                f = fma2(unpack<F16>(v[e]), make_float2(-1.f, -1.f), f);
                                rest[e] = pack<F16>(f.x, f.y);
                            }
                        }
                        *reinterpret_cast<uint4*>(to) = make_uint4(v[0], v[1], v[2], v[3]);
                        if (copy_in_two)
                            *reinterpret_cast<uint4*>(to + rest_at) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                arrive(carry_ready);
            }
            return true;
        };
        // 16 tokens (16 t.. of the half) of 16 channels (16 m.. of the warp's) of
        // chunk c, transposed: a lane has channels lane / 4 and + 8, tokens
        // 2 (lane % 4), + 1 and those + 8
        const int c8 = (KP == 64 ? bw & 1 : bw) * 4 + (lane >> 3 & 1);
        const uint8_t* krow =
            smem + L::OffY + (c8 >> 3) * 16384 + (half * 64 + (lane >> 4) * 8 + (lane & 7)) * 128;
        auto key_tile = [&](int c, int t, int m, uint32_t* x) {
            ldmatrix4_trans(krow + c % L::Stages * L::StageBytes + t * 2048 + ((((c8 + 2 * m) & 7) ^ (lane & 7)) << 4), x);
        };
        // (fp16) the scale of each channel's keys of chunk c: its largest
        // weighted key comes out below 2^15.  A warp has the maxima of its
        // tokens, and exchanges them with the warp of the other tokens.
        auto scale_keys = [&](int c) -> bool {
            const int nv = chunk_n(c);
            if (!wait(&full[c % L::Stages], c / L::Stages)) return false;
            __half2 top[2][2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                top[m][0] = top[m][1] = __float2half2_rn(0.f);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    uint32_t x[4];
                    key_tile(c, t, m, x);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w = x[i] & 0x7fff7fffu;
                        if (nv < kChunk) {
                            const int left = nv - (half * 64 + 16 * t + (i >> 1) * 8 + 2 * (lane & 3));
                            w &= left >= 2 ? 0xffffffffu : left == 1 ? 0xffffu : 0u;
                        }
                        top[m][i & 1] = __hmax2(top[m][i & 1], *reinterpret_cast<const __half2*>(&w));
                    }
                }
            }
            __half* ex = reinterpret_cast<__half*>(smem + L::OffMax) + (c & 1) * kStateWarps * 32;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    __half2 x = top[m][y];
                    x = __hmax2(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = __hmax2(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    if ((lane & 3) == 0) ex[sw * 32 + m * 16 + y * 8 + (lane >> 2)] = __hmax(__low2half(x), __high2half(x));
                }
            arrive(&pair_bar[bw]);
            if (!wait(&pair_bar[bw], c)) return false;
            const float f = fmaxf(__half2float(ex[sw * 32 + lane]), __half2float(ex[(sw ^ 4) * 32 + lane]));
            rs = f < 65536.f ? fp16_scale(f * fabsf(r.key_scale) * fmaxf(1.f, pw[nv])) : 1.f;
            return true;
        };
        // the weighted keys of chunk c
        int kw_n = -1;
        auto weigh_keys = [&](int c) -> bool {
            const int st = c % L::Stages;
            const int nv = chunk_n(c);
            const bool more = c + 1 < nch || want_fin;        // the state behind this chunk is wanted
            uint8_t* base = smem + st * L::StageBytes;
            if (more && nv != kw_n) {
                if (!sync_b()) return false;
                if (ts < 128) kw[ts] = ts < nv ? r.key_scale * pw[rev ? ts + 1 : nv - 1 - ts] : 0.f;
                kw_n = nv;
                if (!sync_b()) return false;
            }
            if (!wait(&full[st], c / L::Stages)) return false;
            // rows behind a packed sequence belong to another one: their
            // values must not meet the zeros of P and the weighted keys
            if (p.cu && nv < kChunk) {
                const int rows = (nv + 15) / 16 * 16 - nv;
                for (int e = ts; e < rows * (VP / 8); e += L::Live * 32) {
                    const int rr = nv + e / (VP / 8), vc = e % (VP / 8);
                    *reinterpret_cast<uint4*>(base + L::OffZ + (vc >> 3) * 16384 + rr * 128 + (vc & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                arrive(z_ready);
            }
            // Parts of the weighted keys of 32 tokens and 16 channels a time,
            // transposed into TMEM: a lane has channels lane / 4 and + 8,
            // tokens 8 i + 2 (lane % 4) and + 1.
            // tokens 32 th.. of the half, both groups of 16 channels: all loads first
            struct Raw {
                uint32_t x[2][8];
                float2 w[4];
            };
            auto raw_keys = [&](int th, Raw& k) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        key_tile(c, 2 * th + t, m, k.x[m] + 4 * t);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    k.w[i] = *reinterpret_cast<const float2*>(kw + half * 64 + 32 * th + 8 * i + 2 * (lane & 3));
            };
            // the first PARTS parts of channels 16 m..
            auto weighted = [&](int m, int th, const Raw& k, uint32_t (&part)[3][8], auto parts) {
                constexpr int PARTS = decltype(parts)::value;
                float2 sc[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float v = F16 ? __shfl_sync(0xffffffffu, rs, m * 16 + y * 8 + (lane >> 2)) : 1.f;
                    sc[y] = make_float2(v, v);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float2 f = mul2(unpack<F16>(k.x[m][2 * i + y]), F16 ? mul2(k.w[i], sc[y]) : k.w[i]);
#pragma unroll
                        for (int q = 0; q < PARTS; ++q) {
                            part[q][2 * i + y] = pack<F16>(f.x, f.y);
                            if (q + 1 < PARTS) f = fma2(unpack<F16>(part[q][2 * i + y]), make_float2(-1.f, -1.f), f);
                        }
                    }
                }
                if (nv < kChunk) {
                    // a select, not the weight 0: what lies behind the end may be inf or NaN
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int left = nv - (half * 64 + 32 * th + 8 * i + 2 * (lane & 3));
                        const uint32_t keep = left >= 2 ? 0xffffffffu : left == 1 ? 0xffffu : 0u;
#pragma unroll
                        for (int q = 0; q < PARTS; ++q) {
                            part[q][2 * i] &= keep;
                            part[q][2 * i + 1] &= keep;
                        }
                    }
                }
            };
            using One = std::integral_constant<int, 1>;
            using Two = std::integral_constant<int, 2>;
            using All = std::integral_constant<int, L::Parts>;
            const uint32_t t_kt = tbase + row + L::Kt + c % L::KtBufs * L::KtCols + half * 32;
            if (more) {
#pragma unroll 1
                for (int th = 0; th < 2; ++th) {
                    Raw k;
                    raw_keys(th, k);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const uint32_t at = t_kt + th * 16 + ((uint32_t)(m * 16) << 16);
                        uint32_t part[3][8];
                        if constexpr (!L::Stacked) {
                            weighted(m, th, k, part, All{});
#pragma unroll
                            for (int q = 0; q < L::KtCols / 64; ++q)
                                tmem_st_16x16(at + q * 64, part[q + (L::Late ? 1 : 0)]);
                        } else if (L::Late) {
                            // the third part, and nothing beside it
                            if (second) {
#pragma unroll
                                for (int j = 0; j < 8; ++j) part[2][j] = 0u;
                            } else {
                                weighted(m, th, k, part, All{});
                            }
                            tmem_st_16x16(at, part[2]);
                        } else if (second) {
                            weighted(m, th, k, part, Two{});
                            tmem_st_16x16(at, part[1]);
                        } else if constexpr (L::KtCols == 128) {
                            weighted(m, th, k, part, All{});
                            tmem_st_16x16(at, part[0]);
                            tmem_st_16x16(at + 64, part[2]);
                        } else {
                            weighted(m, th, k, part, One{});
                            tmem_st_16x16(at, part[0]);
                        }
                    }
                }
            }
            tc_wait_st();
            tc_fence_before();
            arrive(kt_ready(c));
            if constexpr (L::Late) {
                if (more) {
                    if (!wait(bar_kt, c)) return false;
                    tc_fence_after();
#pragma unroll 1
                    for (int th = 0; th < 2; ++th) {
                        Raw k;
                        raw_keys(th, k);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint32_t at = t_kt + th * 16 + ((uint32_t)(m * 16) << 16);
                            uint32_t part[3][8];
                            if (second) {
                                weighted(m, th, k, part, Two{});
                                tmem_st_16x16(at, part[1]);
                            } else {
                                weighted(m, th, k, part, One{});
                                tmem_st_16x16(at, part[0]);
                            }
                        }
                    }
                    tc_wait_st();
                    tc_fence_before();
                    arrive(late_ready);
                }
            }
            return true;
        };
        bool ok = true;
        for (int c = 0; c < nch && ok && live; ++c) {
            if (F16 && (c + 1 < nch || want_fin)) ok = scale_keys(c);
            if (ok) ok = kAhead ? weigh_keys(c) && carry_on(c) : carry_on(c) && weigh_keys(c);
            rs_done = rs;
        }
        if (ok && live && want_fin && seq >= 0 && (nch > 0 || !STATE_ONLY)) {
            if (nch > 0)
                ok = advance(nch - 1);
            else
                initial();
            if constexpr (L::Stacked) {
                // the second half of the rows hands its part of the sum over, in the carry copy's place
                if (ok && !STATE_ONLY && nch > 0) ok = wait(&bar_o[(nch - 1) % NA], (nch - 1) / NA);
                float* sum = reinterpret_cast<float*>(smem + L::OffCarry);      // [VP][64]
                if (ok && second)
#pragma unroll
                    for (int j = 0; j < kCols; ++j) sum[(col0 + j) * 64 + ch] = state[j];
                if (ok) ok = sync_b();
                if (ok && !second)
#pragma unroll
                    for (int j = 0; j < kCols; ++j) state[j] += sum[(col0 + j) * 64 + ch];
            }
            if (ok && ch < r.kd && !second) {
                if constexpr (STATE_ONLY) {
                    float* dst = r.seg + at_seg + ch;
#pragma unroll
                    for (int j = 0; j < kCols; ++j)
                        if (col0 + j < r.vd) dst[(int64_t)(col0 + j) * r.kd] = state[j];
                } else {
                    float* dst = r.fin + at_seq + (int64_t)ch * r.vd + col0;
#pragma unroll
                    for (int j = 0; j < kCols; j += 4)
                        if (col0 + j < r.vd)
                            *reinterpret_cast<float4*>(dst + j) =
                                make_float4(state[j], state[j + 1], state[j + 2], state[j + 3]);
                }
            }
        }
        if (!ok) fail();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == L::MmaWarp) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

// Segment states of split sequences: from each segment's own state (zero
// start) to the state in front of it, in the role's direction of time, and
// the final state.
__global__ void __launch_bounds__(256) la_combine(const __grid_constant__ Params p) {
    const Role& r = p.role[blockIdx.z];
    const int h = blockIdx.x % p.H;
    int seq = blockIdx.x / p.H, len = (int)p.T, sid0 = seq * p.nper, count = p.nper;
    if (p.seqs) {                                             // packed
        const int4 v = p.seqs[seq];
        if (v.x < 0) return;
        seq = v.x;
        sid0 = v.y;
        count = v.z;
        const int start = min(max(p.cu[seq], 0), (int)p.T);
        len = min(max(p.cu[seq + 1], start), (int)p.T) - start;
    }
    // a tile of 32 x 32: a thread has four rows of a column of the segments'
    // states; where the first and the last state lie the other way, they go
    // through shared memory
    const int64_t mat = (int64_t)r.kd * r.vd, at_seq = ((int64_t)seq * p.H + h) * mat;
    const int tiles = (r.kd + 31) / 32, row0 = (int)blockIdx.y % tiles * 32, col0 = (int)blockIdx.y / tiles * 32;
    if (col0 >= r.vd) return;
    __shared__ float turn[32][33];
    const int x4 = threadIdx.x % 8 * 4, y = threadIdx.x / 8;
    const int row = row0 + x4, col = col0 + y;                // of the segments' states
    const int nrow = row0 + y, ncol = col0 + x4;              // of a state in rows
    const bool in = row < r.kd && col < r.vd, nin = nrow < r.kd && ncol < r.vd;
    const float ld = p.log_decay[h];
    const float2 whole = decay_power2(ld, (float)p.seg_len);
    const float tail = decay_power(ld, (float)(len - (count - 1) * p.seg_len));
    const int64_t step = (int64_t)p.H * mat / 4;
    float4* at = reinterpret_cast<float4*>(r.seg + ((int64_t)sid0 * p.H + h) * mat + (int64_t)col * r.kd + row);
    // the last segment's own state is there where the final state is wanted
    const int have = r.fin ? count : count - 1, todo = in ? count : 0;
    // the loads of four segments go out together, the first ones ahead of the
    // initial state's: their addresses do not depend on the running state
    float4 local[4];
    auto fetch = [&](int s) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (in && s + q < have) local[q] = at[(int64_t)(r.rev ? count - 1 - s - q : s + q) * step];
    };
    fetch(0);
    float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r.init && r.init_t) {
        if (in) run = *reinterpret_cast<const float4*>(r.init + at_seq + (int64_t)col * r.kd + row);
    } else if (r.init) {
        if (nin) {
            const float4 v = *reinterpret_cast<const float4*>(r.init + at_seq + (int64_t)nrow * r.vd + ncol);
            turn[y][x4] = v.x;
            turn[y][x4 + 1] = v.y;
            turn[y][x4 + 2] = v.z;
            turn[y][x4 + 3] = v.w;
        }
        __syncthreads();
        run = make_float4(turn[x4][y], turn[x4 + 1][y], turn[x4 + 2][y], turn[x4 + 3][y]);
        __syncthreads();
    }
    for (int s = 0; s < todo; s += 4) {
        if (s) fetch(s);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (s + q >= count) break;
            const int i = r.rev ? count - 1 - s - q : s + q;
            if (s + q > 0 || p.in_place) at[(int64_t)i * step] = run;       // (the first one is init)
            if (s + q < have) {
                const float2 g = i == count - 1 ? make_float2(tail, 0.f) : whole;
                run.x = fmaf(g.x, run.x, fmaf(g.y, run.x, local[q].x));
                run.y = fmaf(g.x, run.y, fmaf(g.y, run.y, local[q].y));
                run.z = fmaf(g.x, run.z, fmaf(g.y, run.z, local[q].z));
                run.w = fmaf(g.x, run.w, fmaf(g.y, run.w, local[q].w));
            }
        }
    }
    if (r.fin) {
        turn[x4][y] = run.x;
        turn[x4 + 1][y] = run.y;
        turn[x4 + 2][y] = run.z;
        turn[x4 + 3][y] = run.w;
        __syncthreads();
        if (nin)
            *reinterpret_cast<float4*>(r.fin + at_seq + (int64_t)nrow * r.vd + ncol) =
                make_float4(turn[y][x4], turn[y][x4 + 1], turn[y][x4 + 2], turn[y][x4 + 3]);
    }
}

__device__ __forceinline__ void used_tokens(const int32_t* cu, int nseq, int64_t T, int64_t& lo, int64_t& hi) {
    lo = min((int64_t)max(cu[0], 0), T);
    hi = min(max((int64_t)cu[nseq], lo), T);
}

// Gradients of shared heads: the fp32 partial results of a group of heads,
// summed in order and rounded once.  rows = B * T; VEC elements a thread.
template <bool F16>
__global__ void __launch_bounds__(256) la_sum_heads(const float* part, uint16_t* out, int64_t rows, int Hx, int rep,
                                                    int D, const int32_t* cu, int nseq) {
    const int64_t per_row = (int64_t)Hx * (D / 4);
    int64_t lo = 0, hi = rows;
    if (cu) used_tokens(cu, nseq, rows, lo, hi);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * per_row; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per_row, x = i % per_row;
        const int hx = (int)(x / (D / 4)), d = (int)(x % (D / 4)) * 4;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row >= lo && row < hi) {
            const float* src = part + (row * Hx * rep + (int64_t)hx * rep) * D + d;
            for (int j = 0; j < rep; ++j) {
                const float4 v = *reinterpret_cast<const float4*>(src + (int64_t)j * D);
                sum.x += v.x;
                sum.y += v.y;
                sum.z += v.z;
                sum.w += v.w;
            }
        }
        uint2 v;
        v.x = pack<F16>(sum.x, sum.y);
        v.y = pack<F16>(sum.z, sum.w);
        *reinterpret_cast<uint2*>(out + (row * Hx + hx) * D + d) = v;
    }
}

// Zero the rows of tokens that no packed sequence holds.
__global__ void __launch_bounds__(256) la_zero_rest(uint16_t* out, int64_t T, int H, int D, int64_t st, int64_t sh,
                                                    const int32_t* cu, int nseq) {
    int64_t lo, hi;
    used_tokens(cu, nseq, T, lo, hi);
    const int64_t per_row = (int64_t)H * (D / 8), count = (lo + T - hi) * per_row;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
        int64_t t = i / per_row;
        const int64_t x = i % per_row;
        if (t >= lo) t += hi - lo;
        *reinterpret_cast<uint4*>(out + t * st + x / (D / 8) * sh + x % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
    }
}

// ------------------------------------------------------------------ host ---

int fail(int status, const std::string& msg) {
    set_last_error(msg.c_str());
    return status;
}
int cuda_fail(cudaError_t e, const char* what) {
    (void)cudaGetLastError();                                 // (reported here, and not by the next call too)
    return fail(FFTCONV_ERR_CUDA, std::string(what) + ": " + cudaGetErrorName(e) + " (" + cudaGetErrorString(e) + ")");
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult got;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &got) !=
                cudaSuccess ||
            got != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

// [B, T, H, D] with element strides: tiles of `tokens` x 128 bytes of one
// head, in the 128-byte swizzle; what lies outside reads as zero and is not
// written.
int make_map(CUtensorMap* m, const void* base, int dtype, int64_t B, int64_t T, int64_t H, int64_t D,
             const int64_t* stride, int tokens = kChunk) {
    // the encoder is a driver call: it needs the device's context bound to
    // this thread, which autograd's threads have not done before their first
    // runtime call
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess)
        return fail(FFTCONV_ERR_CUDA, "no current device");
    const EncodeTiled fn = encode_tiled();
    if (!fn) return fail(FFTCONV_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T, (cuuint64_t)B};
    const int size = dtype == FFTCONV_F32 ? 4 : 2;
    auto bytes = [&](int64_t extent, int64_t s) { return (cuuint64_t)(extent > 1 ? s * size : 16); };
    const cuuint64_t strides[3] = {bytes(H, stride[2]), bytes(T, stride[1]), bytes(B, stride[0])};
    const cuuint32_t box[4] = {(cuuint32_t)(128 / size), 1, (cuuint32_t)tokens, 1}, one[4] = {1, 1, 1, 1};
    const CUresult e = fn(m,
                          dtype == FFTCONV_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                          : dtype == FFTCONV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                          4, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (e != CUDA_SUCCESS) return fail(FFTCONV_ERR_CUDA, "cuTensorMapEncodeTiled failed: " + std::to_string((int)e));
    return FFTCONV_OK;
}

int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 148;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <int KP, int VP, bool F16, bool STATE_ONLY, bool EXACT, bool FINE>
cudaError_t launch(const Params& p, int64_t ctas, cudaStream_t s) {
    using L = Layout<KP, VP, F16, STATE_ONLY, EXACT>;
    static std::atomic<uint64_t> ready{0};                    // devices whose kernel has its shared memory size
    auto* kern = la_kernel<KP, VP, F16, STATE_ONLY, EXACT, FINE>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !((ready.load(std::memory_order_relaxed) >> dev) & 1)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::Bytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
    void* args[] = {const_cast<Params*>(&p)};
    return cudaLaunchKernel(reinterpret_cast<const void*>(kern), dim3((unsigned)ctas), dim3(L::Threads), args, L::Bytes,
                            s);
}

template <int KP, int VP, bool STATE_ONLY, bool FINE>
cudaError_t launch_type(const Params& p, bool f16, bool exact, int64_t ctas, cudaStream_t s) {
    // (128 channels in fp16 have two parts either way)
    if (f16)
        return exact && KP == 64 ? launch<KP, VP, true, STATE_ONLY, KP == 64, FINE>(p, ctas, s)
                                 : launch<KP, VP, true, STATE_ONLY, false, FINE>(p, ctas, s);
    return exact ? launch<KP, VP, false, STATE_ONLY, true, FINE>(p, ctas, s)
                 : launch<KP, VP, false, STATE_ONLY, false, FINE>(p, ctas, s);
}

template <bool STATE_ONLY, bool FINE>
cudaError_t launch_kernel(const Params& p, bool f16, bool exact, int kp, int vp, int64_t ctas, cudaStream_t s) {
    if (kp == 64)
        return vp == 64 ? launch_type<64, 64, STATE_ONLY, FINE>(p, f16, exact, ctas, s)
                        : launch_type<64, 128, STATE_ONLY, FINE>(p, f16, exact, ctas, s);
    return vp == 64 ? launch_type<128, 64, STATE_ONLY, FINE>(p, f16, exact, ctas, s)
                    : launch_type<128, 128, STATE_ONLY, FINE>(p, f16, exact, ctas, s);
}

// Calls of up to so many tokens have P in two parts.  A row of a short prompt
// is one term or a few, and all channels of the output share the rounding of
// its P: with one part, prompts of 1 to 20 tokens were up to 1.75 times as far
// from the exact outputs as a form that rounds these only, over many rows
// sqrt(2) times.  It costs the second products and a tenth of a long walk
// (16 x 4096 tokens, 12 heads of 64/64, both passes at the power limit: 435 us
// with one part and 475 with two), and less of a short call (16 heads, one
// part and two: 37 tokens 8.7 us either way, 8 x 256 tokens of 128/128 bf16
// 18.8 and 19.0, 2 x 1024 of them fp16, both passes, 95.0 and 102.4).
constexpr int64_t kFineTokens = 2048;

// How a call's sequences are cut into segments, one CTA for each (segment,
// head, role).
struct Split {
    int64_t seg_len, nper, max_seg;           // nper: segments of a sequence (unpacked)
    int64_t max_cut, max_seqs;                // segments of cut sequences (those with states in the workspace), cut sequences
    bool on;
};

// A sequence is one CTA's serial walk, so few sequences x heads leave SMs
// idle; cutting along time costs a second pass over keys and values (the
// segments' own states) and the states' round trip.  It pays where one walk
// takes over 1.6 times what an even share of all tokens would (bf16, forward:
// at 1.54 times, 16 x 4096 tokens, 12 heads of 64/64, 117 us and 142 cut; 12 x
// 4096, 8 heads of 128/128, 118 and 157; at 2.05 times, 8 x 4096, 9 heads of
// 128/128, 115 and 99 cut; 64/64 61 and 60).
Split split_of(const fftconv_linear_attention_t& d, int nroles) {
    const int64_t sms = sm_count(), seqs = d.nseq > 0 ? d.nseq : d.B;
    const int64_t tasks = seqs * d.H * nroles;
    auto up = [](int64_t x) { return (x + kChunk - 1) / kChunk * kChunk; };
    Split s{up(d.T), 1, seqs, 0, 0, false};
    int64_t len;
    if (d.nseq > 0) {
        // lengths are known on the device only.  Pieces a little longer than
        // an even share leave room for the sequences' short ends beside them
        // (us with pieces of 3/4 of a share, one, 5/4 and 3/2, in a graph:
        // 8192 tokens in 9 sequences, 16 heads of 128/128 88 79 73 83, both
        // passes 230 204 213 222; 32768 in 40, 12 heads of 64/64 135 148 122
        // 134; 16384 in 5, 8 heads of 64/64 77 57 60 67; 16384 in 12, 4 heads
        // of 128/128 fp16 52 52 59 62; 65536 in 30, 6 heads of 64/64, both
        // passes 260 224 223 251)
        len = up((d.T * d.H * nroles * 5 / 4 + sms - 1) / sms);
    } else {
        const int64_t share = (d.B * d.T * d.H * nroles + sms - 1) / sms;
        if (d.T * ((tasks + sms - 1) / sms) <= share + share * 3 / 5 + 4 * kChunk) return s;
        const int64_t pieces = sms / tasks < 2 ? 2 : sms / tasks;
        len = up((d.T + pieces - 1) / pieces);
    }
    if (len < 4 * kChunk) len = 4 * kChunk;
    if (len >= d.T) return s;
    s.seg_len = len;
    s.nper = (d.T + len - 1) / len;
    s.max_seg = d.nseq > 0 ? d.T / len + d.nseq : d.B * s.nper;
    // (more than one segment: over len tokens, and fewer than 2 n / len segments of n)
    s.max_cut = d.nseq > 0 && 2 * d.T / len < s.max_seg ? 2 * d.T / len : s.max_seg;
    s.max_seqs = d.nseq > 0 && d.T / len < seqs ? d.T / len : seqs;
    s.on = true;
    return s;
}

int64_t pad256(int64_t b) { return (b + 255) / 256 * 256; }

int check_shape(const fftconv_linear_attention_t* d) {
    if (!d) return fail(FFTCONV_ERR_INVALID_ARG, "shape is NULL");
    if (d->B < 0 || d->T < 0 || d->nseq < 0) return fail(FFTCONV_ERR_INVALID_ARG, "B, T or nseq is negative");
    if (d->H <= 0 || d->Hq <= 0 || d->Hk <= 0 || d->Hv <= 0 || d->H % d->Hq || d->H % d->Hk || d->H % d->Hv)
        return fail(FFTCONV_ERR_INVALID_ARG, "Hq, Hk and Hv must be positive and divide H");
    if (d->dtype != FFTCONV_F16 && d->dtype != FFTCONV_BF16)
        return fail(d->dtype == FFTCONV_F32 ? FFTCONV_ERR_UNSUPPORTED : FFTCONV_ERR_INVALID_ARG,
                    "linear attention takes fp16 or bf16 tensors");
    if (d->K <= 0 || d->V <= 0) return fail(FFTCONV_ERR_INVALID_ARG, "K and V must be positive");
    if (d->K % 8 || d->V % 8 || d->K > 128 || d->V > 128)
        return fail(FFTCONV_ERR_UNSUPPORTED, "K and V must be multiples of 8 up to 128");
    if (d->nseq > 0 && d->B != 1) return fail(FFTCONV_ERR_INVALID_ARG, "packed sequences need B = 1");
    if (d->T >= (int64_t(1) << 31) - 256 || d->B >= (int64_t(1) << 31) || d->H >= 65536 || d->nseq >= (1 << 24))
        return fail(FFTCONV_ERR_UNSUPPORTED, "B, T, H or nseq too large");
    const double seqs = d->nseq > 0 ? (double)d->nseq : (double)d->B;
    if (seqs * (double)d->H * 3.0 + (double)d->B * (double)d->T * (double)d->H * 3.0 / 512.0 >= 2147483647.0)
        return fail(FFTCONV_ERR_UNSUPPORTED, "too many sequences and heads for one launch");
    return FFTCONV_OK;
}

int check_stride(const char* name, const int64_t* s, int64_t B, int64_t T, int64_t H) {
    const int64_t extent[3] = {B, T, H};
    for (int i = 0; i < 3; ++i)
        if (extent[i] > 1 && (s[i] <= 0 || s[i] % 8 || s[i] >= (int64_t(1) << 38)))
            return fail(FFTCONV_ERR_ALIGNMENT,
                        std::string(name) + ": strides must be positive multiples of 8 elements (16 bytes)");
    return FFTCONV_OK;
}

// The elements a strided tensor spans.
int64_t span(const int64_t* s, int64_t B, int64_t T, int64_t H, int64_t D) {
    return (B - 1) * (B > 1 ? s[0] : 0) + (T - 1) * (T > 1 ? s[1] : 0) + (H - 1) * (H > 1 ? s[2] : 0) + D;
}
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
    if (!a || !b || na <= 0 || nb <= 0) return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// la_plan's tables
int64_t plan_bytes(const Split& s) {
    return pad256(s.max_seg * 2 * sizeof(int4)) + pad256(s.max_cut * 2 * sizeof(int4)) +
           pad256(s.max_seqs * sizeof(int4));
}
// the segments' states of a role
int64_t state_bytes(const fftconv_linear_attention_t& d, const Split& s) {
    return pad256(s.max_cut * d.H * d.K * d.V * 4);
}

size_t workspace_bytes(const fftconv_linear_attention_t& d, bool backward) {
    if (d.B == 0 || d.T == 0) return 0;
    const int nroles = backward ? 3 : 1;
    const Split s = split_of(d, nroles);
    int64_t n = 0;
    if (s.on) n += nroles * state_bytes(d, s);
    if (s.on && d.nseq > 0) n += plan_bytes(s);
    if (backward) {
        if (d.Hq < d.H) n += pad256(d.T * d.B * d.H * d.K * 4);
        if (d.Hk < d.H) n += pad256(d.T * d.B * d.H * d.K * 4);
        if (d.Hv < d.H) n += pad256(d.T * d.B * d.H * d.V * 4);
    }
    return (size_t)n;
}

void fill(Params& p, const fftconv_linear_attention_t& d, const Split& s, const float* log_decay, const int32_t* cu,
          int nroles) {
    p.log_decay = log_decay;
    p.cu = d.nseq > 0 ? cu : nullptr;
    p.T = d.T;
    p.nroles = nroles;
    p.H = (int)d.H;
    p.nseq = (int)d.nseq;
    p.nper = (int)s.nper;
    p.seg_len = (int)s.seg_len;
    p.max_seg = (int)s.max_seg;
    p.max_cut = (int)s.max_cut;
    p.max_seqs = (int)s.max_seqs;
    p.in_place = 0;
}

// The tables of packed sequences that may be cut, at ws.
cudaError_t plan(Params& p, const fftconv_linear_attention_t& d, const Split& s, uint8_t* ws, cudaStream_t stream) {
    if (!s.on || d.nseq == 0) return cudaSuccess;
    p.table = reinterpret_cast<int4*>(ws);
    p.cuts = reinterpret_cast<int4*>(ws + pad256(s.max_seg * 2 * sizeof(int4)));
    p.seqs = reinterpret_cast<int4*>((uint8_t*)p.cuts + pad256(s.max_cut * 2 * sizeof(int4)));
    la_plan<<<1, d.nseq < 1024 ? (unsigned)(d.nseq + 31) / 32 * 32 : 1024, 0, stream>>>(p);
    return cudaGetLastError();
}

// The launches of up to three roles, all with key and value dims within
// (kp, vp).
cudaError_t run_roles(const Params& p, const fftconv_linear_attention_t& d, const Split& s, int kp, int vp,
                      cudaStream_t stream) {
    const bool f16 = d.dtype == FFTCONV_F16;
    const int64_t ctas = s.max_seg * d.H * p.nroles;
    bool exact = false;                       // a state is a result
    for (int i = 0; i < p.nroles; ++i) exact |= p.role[i].fin != nullptr;
    if (s.on) {
        cudaError_t e = launch_kernel<true, false>(p, f16, exact, kp, vp, s.max_cut * d.H * p.nroles, stream);
        if (e != cudaSuccess) return e;
        void* args[] = {const_cast<Params*>(&p)};
        e = cudaLaunchKernel(reinterpret_cast<const void*>(la_combine),
                             dim3((unsigned)(s.max_seqs * d.H), (unsigned)((d.K + 31) / 32 * ((d.V + 31) / 32)), (unsigned)p.nroles),
                             dim3(256), args, 0, stream);
        if (e != cudaSuccess) return e;
    }
    // (packed sequences that are not cut take their final state from this
    // launch, all of which then runs the exact form.  With their states from
    // the launch before it 8192 tokens in 9 sequences took 90 us instead of
    // 95, but 2048 sequences of 64 tokens 2730 instead of 1870.)
    exact &= !s.on || p.cu;
    return d.B * d.T <= kFineTokens ? launch_kernel<false, true>(p, f16, exact, kp, vp, ctas, stream)
                                    : launch_kernel<false, false>(p, f16, exact, kp, vp, ctas, stream);
}

cudaError_t copy_states(float* dst, const float* src, int64_t count, cudaStream_t s) {
    if (!dst || !count || dst == src) return cudaSuccess;
    if (src) return cudaMemcpyAsync(dst, src, (size_t)count * 4, cudaMemcpyDeviceToDevice, s);
    return cudaMemsetAsync(dst, 0, (size_t)count * 4, s);
}

cudaError_t zero_rest(void* out, const fftconv_linear_attention_t& d, int64_t H, int64_t D, const int64_t* st,
                      const int32_t* cu, cudaStream_t s) {
    const int64_t blocks = (d.T * H * D / 8 + 255) / 256;
    la_zero_rest<<<(unsigned)(blocks < 592 ? blocks : 592), 256, 0, s>>>((uint16_t*)out, d.T, (int)H, (int)D, st[1],
                                                                        st[2], cu, (int)d.nseq);
    return cudaGetLastError();
}

}  // namespace
}  // namespace fftconv

using namespace fftconv;

extern "C" {

size_t fftconv_linear_attention_workspace_bytes(const fftconv_linear_attention_t* shape, int backward) {
    if (check_shape(shape) != FFTCONV_OK) return 0;
    return workspace_bytes(*shape, backward != 0);
}

int fftconv_linear_attention(const fftconv_linear_attention_t* shape, const void* q, const void* k, const void* v,
                             const float* log_decay, const float* initial_state, const int32_t* cu_seqlens, void* o,
                             float* final_state, void* workspace, size_t workspace_size, fftconv_stream_t stream) {
    set_last_error("");
    if (int e = check_shape(shape)) return e;
    const fftconv_linear_attention_t& d = *shape;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t seqs = d.nseq > 0 ? d.nseq : d.B, states = seqs * d.H * d.K * d.V;
    if (d.nseq > 0 && !cu_seqlens) return fail(FFTCONV_ERR_INVALID_ARG, "cu_seqlens is NULL");
    if (d.nseq == 0 && cu_seqlens) return fail(FFTCONV_ERR_INVALID_ARG, "cu_seqlens given with nseq = 0");
    if (seqs == 0) return FFTCONV_OK;
    if (!log_decay) return fail(FFTCONV_ERR_INVALID_ARG, "log_decay is NULL");
    if (!aligned16(initial_state) || !aligned16(final_state))
        return fail(FFTCONV_ERR_ALIGNMENT, "states must be 16-byte aligned");
    if (final_state != initial_state && overlap(final_state, states * 4, initial_state, states * 4))
        return fail(FFTCONV_ERR_INVALID_ARG, "final_state overlaps initial_state");
    if (d.T == 0) {
        const cudaError_t e = copy_states(final_state, initial_state, states, s);
        return e == cudaSuccess ? FFTCONV_OK : cuda_fail(e, "state copy");
    }
    if (!q || !k || !v || !o) return fail(FFTCONV_ERR_INVALID_ARG, "q, k, v and o must be non-NULL");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o))
        return fail(FFTCONV_ERR_ALIGNMENT, "q, k, v and o must be 16-byte aligned");
    if (int e = check_stride("q", d.q_stride, d.B, d.T, d.Hq)) return e;
    if (int e = check_stride("k", d.k_stride, d.B, d.T, d.Hk)) return e;
    if (int e = check_stride("v", d.v_stride, d.B, d.T, d.Hv)) return e;
    if (int e = check_stride("o", d.o_stride, d.B, d.T, d.H)) return e;
    const int64_t no = span(d.o_stride, d.B, d.T, d.H, d.V) * 2;
    if (overlap(o, no, q, span(d.q_stride, d.B, d.T, d.Hq, d.K) * 2) ||
        overlap(o, no, k, span(d.k_stride, d.B, d.T, d.Hk, d.K) * 2) ||
        overlap(o, no, v, span(d.v_stride, d.B, d.T, d.Hv, d.V) * 2) || overlap(o, no, initial_state, states * 4) ||
        overlap(o, no, final_state, states * 4))
        return fail(FFTCONV_ERR_INVALID_ARG, "o overlaps another tensor");
    const Split sp = split_of(d, 1);
    const size_t need = workspace_bytes(d, false);
    if (need && (!workspace || workspace_size < need))
        return fail(FFTCONV_ERR_INVALID_ARG, "workspace of " + std::to_string(workspace_size) + " bytes, " +
                                                 std::to_string(need) + " needed");
    if (need && (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return fail(FFTCONV_ERR_ALIGNMENT, "workspace not 256-byte aligned");

    (void)cudaGetLastError();                                 // (an earlier call's error is not this one's)
    Params p{};
    fill(p, d, sp, log_decay, cu_seqlens, 1);
    if (int e = make_map(&p.maps[0], q, d.dtype, d.B, d.T, d.Hq, d.K, d.q_stride)) return e;
    if (int e = make_map(&p.maps[1], k, d.dtype, d.B, d.T, d.Hk, d.K, d.k_stride)) return e;
    if (int e = make_map(&p.maps[2], v, d.dtype, d.B, d.T, d.Hv, d.V, d.v_stride)) return e;
    if (int e = make_map(&p.maps[3], o, d.dtype, d.B, d.T, d.H, d.V, d.o_stride, 32)) return e;
    Role& r = p.role[0];
    r.x = 0; r.y = 1; r.z = 2;
    r.out_map = 3;
    r.x_div = (int)(d.H / d.Hq); r.y_div = (int)(d.H / d.Hk); r.z_div = (int)(d.H / d.Hv);
    r.kd = (int)d.K; r.vd = (int)d.V;
    r.a_in = r.a_carry = d.scale;
    r.key_scale = 1.f;
    r.out = o;
    r.out_b = d.o_stride[0]; r.out_t = d.o_stride[1]; r.out_h = d.o_stride[2];
    r.init = initial_state;
    r.fin = final_state;
    r.seg = (float*)workspace;
    p.in_place = sp.on && initial_state && final_state == initial_state;
    cudaError_t e = cudaSuccess;
    if (d.nseq > 0 && d.zero_rest) e = zero_rest(o, d, d.H, d.V, d.o_stride, cu_seqlens, s);
    if (e == cudaSuccess) e = plan(p, d, sp, (uint8_t*)workspace + state_bytes(d, sp), s);
    if (e == cudaSuccess) e = run_roles(p, d, sp, d.K > 64 ? 128 : 64, d.V > 64 ? 128 : 64, s);
    return e == cudaSuccess ? FFTCONV_OK : cuda_fail(e, "linear attention launch");
}

int fftconv_linear_attention_backward(const fftconv_linear_attention_t* shape, const void* q, const void* k,
                                      const void* v, const float* log_decay, const float* initial_state,
                                      const int32_t* cu_seqlens, const void* do_, const float* dfinal, void* dq,
                                      void* dk, void* dv, float* dinitial, void* workspace, size_t workspace_size,
                                      fftconv_stream_t stream) {
    set_last_error("");
    if (int e = check_shape(shape)) return e;
    const fftconv_linear_attention_t& d = *shape;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t seqs = d.nseq > 0 ? d.nseq : d.B, states = seqs * d.H * d.K * d.V;
    if (d.nseq > 0 && !cu_seqlens) return fail(FFTCONV_ERR_INVALID_ARG, "cu_seqlens is NULL");
    if (d.nseq == 0 && cu_seqlens) return fail(FFTCONV_ERR_INVALID_ARG, "cu_seqlens given with nseq = 0");
    if (seqs == 0) return FFTCONV_OK;
    if (!log_decay) return fail(FFTCONV_ERR_INVALID_ARG, "log_decay is NULL");
    if (!aligned16(initial_state) || !aligned16(dfinal) || !aligned16(dinitial))
        return fail(FFTCONV_ERR_ALIGNMENT, "states must be 16-byte aligned");
    if (overlap(dinitial, states * 4, dfinal, states * 4))
        return fail(FFTCONV_ERR_INVALID_ARG, "dinitial overlaps dfinal");
    if (d.T == 0) {
        const cudaError_t e = copy_states(dinitial, dfinal, states, s);
        return e == cudaSuccess ? FFTCONV_OK : cuda_fail(e, "state copy");
    }
    if (!q || !k || !v || !do_ || !dq || !dk || !dv)
        return fail(FFTCONV_ERR_INVALID_ARG, "q, k, v, do_, dq, dk and dv must be non-NULL");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(do_) || !aligned16(dq) || !aligned16(dk) ||
        !aligned16(dv))
        return fail(FFTCONV_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
    if (int e = check_stride("q", d.q_stride, d.B, d.T, d.Hq)) return e;
    if (int e = check_stride("k", d.k_stride, d.B, d.T, d.Hk)) return e;
    if (int e = check_stride("v", d.v_stride, d.B, d.T, d.Hv)) return e;
    if (int e = check_stride("do_", d.o_stride, d.B, d.T, d.H)) return e;
    const int64_t tok = d.B * d.T;
    {
        const void* in[6] = {q, k, v, do_, initial_state, dfinal};
        const int64_t nin[6] = {span(d.q_stride, d.B, d.T, d.Hq, d.K) * 2, span(d.k_stride, d.B, d.T, d.Hk, d.K) * 2,
                                span(d.v_stride, d.B, d.T, d.Hv, d.V) * 2, span(d.o_stride, d.B, d.T, d.H, d.V) * 2,
                                states * 4, states * 4};
        const void* out[4] = {dq, dk, dv, dinitial};
        const int64_t nout[4] = {tok * d.Hq * d.K * 2, tok * d.Hk * d.K * 2, tok * d.Hv * d.V * 2, states * 4};
        for (int i = 0; i < 4; ++i) {
            for (int j = 0; j < 6; ++j)
                if (overlap(out[i], nout[i], in[j], nin[j]))
                    return fail(FFTCONV_ERR_INVALID_ARG, "a gradient overlaps an input");
            for (int j = 0; j < i; ++j)
                if (overlap(out[i], nout[i], out[j], nout[j]))
                    return fail(FFTCONV_ERR_INVALID_ARG, "two gradients overlap");
        }
    }
    const Split sp = split_of(d, 3);
    const size_t need = workspace_bytes(d, true);
    if (need && (!workspace || workspace_size < need))
        return fail(FFTCONV_ERR_INVALID_ARG, "workspace of " + std::to_string(workspace_size) + " bytes, " +
                                                 std::to_string(need) + " needed");
    if (need && (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return fail(FFTCONV_ERR_ALIGNMENT, "workspace not 256-byte aligned");

    uint8_t* ws = (uint8_t*)workspace;
    auto take = [&](int64_t bytes) {
        uint8_t* at = ws;
        ws += pad256(bytes);
        return at;
    };
    float* seg[3] = {nullptr, nullptr, nullptr};
    if (sp.on)
        for (int i = 0; i < 3; ++i) seg[i] = (float*)take(state_bytes(d, sp));
    uint8_t* const table = sp.on && d.nseq > 0 ? take(plan_bytes(sp)) : nullptr;
    float* part[3] = {nullptr, nullptr, nullptr};
    if (d.Hq < d.H) part[0] = (float*)take(tok * d.H * d.K * 4);
    if (d.Hk < d.H) part[1] = (float*)take(tok * d.H * d.K * 4);
    if (d.Hv < d.H) part[2] = (float*)take(tok * d.H * d.V * 4);

    (void)cudaGetLastError();                                 // (an earlier call's error is not this one's)
    Params p{};
    fill(p, d, sp, log_decay, cu_seqlens, 3);
    if (int e = make_map(&p.maps[0], q, d.dtype, d.B, d.T, d.Hq, d.K, d.q_stride)) return e;
    if (int e = make_map(&p.maps[1], k, d.dtype, d.B, d.T, d.Hk, d.K, d.k_stride)) return e;
    if (int e = make_map(&p.maps[2], v, d.dtype, d.B, d.T, d.Hv, d.V, d.v_stride)) return e;
    if (int e = make_map(&p.maps[3], do_, d.dtype, d.B, d.T, d.H, d.V, d.o_stride)) return e;
    const int div[4] = {(int)(d.H / d.Hq), (int)(d.H / d.Hk), (int)(d.H / d.Hv), 1};
    void* out[3] = {dq, dk, dv};
    const int64_t heads[3] = {d.Hq, d.Hk, d.Hv}, dims[3] = {d.K, d.K, d.V};
    const int sides[3][3] = {{3, 2, 1}, {2, 3, 0}, {1, 0, 3}};
    for (int i = 0; i < 3; ++i) {
        Role& r = p.role[i];
        r.x = sides[i][0]; r.y = sides[i][1]; r.z = sides[i][2];
        r.x_div = div[r.x]; r.y_div = div[r.y]; r.z_div = div[r.z];
        r.rev = i > 0;
        r.kd = (int)(i < 2 ? d.V : d.K);
        r.vd = (int)dims[i];
        r.a_in = d.scale;
        r.a_carry = i == 0 ? d.scale : 1.f;
        r.key_scale = i == 0 ? 1.f : d.scale;
        r.init = i == 0 ? initial_state : dfinal;
        r.init_t = i < 2;
        r.fin = i == 2 ? dinitial : nullptr;
        r.seg = seg[i];
        r.out_f32 = part[i] != nullptr;
        r.out = part[i] ? (void*)part[i] : out[i];
        const int64_t hh = part[i] ? d.H : heads[i];
        r.out_h = dims[i];
        r.out_t = hh * dims[i];
        r.out_b = d.T * hh * dims[i];
        r.out_map = 4 + i;
        const int64_t st[3] = {r.out_b, r.out_t, r.out_h};
        if (int e = make_map(&p.maps[4 + i], r.out, part[i] ? (int)FFTCONV_F32 : d.dtype, d.B, d.T, hh, dims[i], st, 32))
            return e;
    }
    cudaError_t e = cudaSuccess;
    if (d.nseq > 0)
        for (int i = 0; i < 3 && e == cudaSuccess; ++i) {
            const int64_t st[3] = {0, heads[i] * dims[i], dims[i]};
            if (!part[i]) e = zero_rest(out[i], d, heads[i], dims[i], st, cu_seqlens, s);
        }
    if (e == cudaSuccess) e = plan(p, d, sp, table, s);
    if (e == cudaSuccess) {
        const int kp = d.K > 64 ? 128 : 64, vp = d.V > 64 ? 128 : 64;
        // Mixed widths: one launch at the larger one where that saves enough
        // waves of CTAs over two in a row, whose waves are a sixth shorter
        // (2048 tokens, heads of 128/64, bf16, one launch and two: 48
        // sequences x heads 91 and 104 us, 72 119 and 109, 96 130 and 162)
        const int64_t sms = sm_count(), n = sp.max_seg * d.H;
        auto waves = [&](int64_t ctas) { return (ctas + sms - 1) / sms; };
        if (kp == vp || waves(3 * n) * 6 <= (waves(2 * n) + waves(n)) * 5) {
            const int w = kp > vp ? kp : vp;
            e = run_roles(p, d, sp, w, w, s);
        } else {
            // dq and dk have the dims (V, K), dv has (K, V)
            Params a = p;
            a.nroles = 2;
            e = run_roles(a, d, sp, vp, kp, s);
            if (e == cudaSuccess) {
                a.nroles = 1;
                a.role[0] = p.role[2];
                e = run_roles(a, d, sp, kp, vp, s);
            }
        }
    }
    for (int i = 0; i < 3 && e == cudaSuccess; ++i) {
        if (!part[i]) continue;
        const int64_t work = (tok * heads[i] * (dims[i] / 4) + 255) / 256;
        const unsigned grid = (unsigned)(work < 148 * 32 ? work : 148 * 32);
        const int rep = (int)(d.H / heads[i]);
        const int32_t* cu = d.nseq > 0 ? cu_seqlens : nullptr;
        if (d.dtype == FFTCONV_F16)
            la_sum_heads<true><<<grid, 256, 0, s>>>(part[i], (uint16_t*)out[i], tok, (int)heads[i], rep, (int)dims[i],
                                                    cu, (int)d.nseq);
        else
            la_sum_heads<false><<<grid, 256, 0, s>>>(part[i], (uint16_t*)out[i], tok, (int)heads[i], rep,
                                                     (int)dims[i], cu, (int)d.nseq);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? FFTCONV_OK : cuda_fail(e, "linear attention backward launch");
}

int fftconv_linear_attention_status(fftconv_stream_t stream) {
    set_last_error("");
    cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
    int st = 0;
    const int zero = 0;
    if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(&st, g_status, sizeof(int), 0, cudaMemcpyDeviceToHost, (cudaStream_t)stream);
    if (e == cudaSuccess) e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, (cudaStream_t)stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "linear attention status");
    return st;
}

}  // extern "C"
