// ops_rows.cuh -- the row kernels: activation rows to 8-bit codes (plain,
// gathered, SwiGLU'd, or a weighted sum of expert rows), and the norms before
// and after a block.
//
// All are one pass over memory: a CTA owns a row at a time (grid-strided), takes
// the row's reductions (sum of squares, largest magnitude) by warp shuffles and
// one shared-memory exchange each, and writes the outputs.  What bounds them is
// HBM traffic for many rows and launch-to-finish latency for one.
//
//  k_pipe   rows whose pieces are 16-byte aligned, up to 12288 values: each
//           thread copies its own pieces of the next rows into shared memory
//           asynchronously (cp.async, no barrier needed to read them back) while
//           it works on the current one, and the norms' weights once per CTA.
//  k_rows   the rest: the weighted combine (its k rows a token are already that
//           many independent loads), unaligned rows (element by element), and
//           aligned ones past k_pipe's length.  Rows longer than a CTA's registers
//           hold (16384 values) take the same steps but read their inputs again
//           for each, as do aligned rows where that is quicker.
//
// Measured on B200: 8192 x 4096 bf16 to codes 21 us (4.8 TB/s), 16384 gathered rows
// of 1792 22.6, SwiGLU of 16384 x 2048 19.7 (4.3 TB/s), norm of 2048 x 4096 bf16 12,
// residual norm with the next norm 18.1 (3.7 TB/s); one row of 4096 2.6 to 5 us.  What
// keeps many rows from HBM speed is instruction issue for codes, and for the norms
// latency: 12 warps an SM, two dependent reductions a row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/elq_ops.h"
#include "../csrc/elq_device.cuh"

namespace elqops {

using elq::pdl_trigger;
using elq::pdl_wait;

enum RowOp { ROW_QUANT = 0, ROW_SWIGLU = 1, ROW_COMBINE = 2, ROW_RMS = 3, ROW_RESIDUAL = 4 };

struct RowArgs {
    int64_t rows;
    int cols;
    // sources: x (x, gu, o, or the y of a residual norm); h the residual stream
    const void* x;
    int x_type;
    int64_t ldx, x_rows;
    const void* h;
    int64_t ldh;
    const int32_t* index;       // row indices (quantise) or positions (combine)
    int div, k;
    const float* weights;       // combine
    const float* w;             // norm weight (rms: of n; residual: of y)
    const float* gate;
    int64_t gate_rows, gate_ld;
    int gate_cols;
    const float* w_next;
    float res_scale, eps, inv_cols;
    // outputs
    void* h_out;
    int h_type;
    int64_t ld_out;
    void* n;                    // codes, or the normalised row
    int n_type;
    int64_t ldn;
    float* scale;
    // k_pipe: what a CTA keeps in shared memory
    int w_planes, row_planes;   // 16-byte pieces a thread's chunk has of the weights, and of a row
};

constexpr int kRowThreads = 512;        // most threads of a CTA

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Eight 16-bit values.
__device__ __forceinline__ void widen8(const uint4& r, int type, float (&v)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    // one branch for all eight, not a choice between two conversions of each
    if (type == ELQ_BF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = bf16_lo(w[j]);
            v[2 * j + 1] = bf16_hi(w[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
        }
    }
}

__device__ __forceinline__ void store1(void* p, int type, int64_t i, float v) {
    if (type == ELQ_F32) reinterpret_cast<float*>(p)[i] = v;
    else if (type == ELQ_BF16) reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void store8(void* p, int type, int64_t i, const float (&v)[8]) {
    if (type == ELQ_F32) {
        float4* d = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
        d[0] = make_float4(v[0], v[1], v[2], v[3]);
        d[1] = make_float4(v[4], v[5], v[6], v[7]);
        return;
    }
    uint4* d = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i);
    if (type == ELQ_BF16)
        *d = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    else
        *d = make_uint4(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]), pack_f16(v[4], v[5]), pack_f16(v[6], v[7]));
}

// Pairs of fp32 values in one 64-bit register, and the packed operations on them:
// each half is one IEEE round-to-nearest operation, at half the instructions.
typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 halves(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 sub2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// The largest of three magnitudes, a NaN if one is a NaN.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The scale of a row and what its codes need: x / s to the nearest whole
// number, exactly.  q = rint(x * inv) is within one of it; the remainder
// r = x - q * s is exact in fp32 (one fused multiply-add), and its comparison
// with s / 2 settles the rounding, halves away from zero.  A scale below 2^-100
// is worked on times 2^100 (exact) so that its reciprocal is finite.
struct CodeScale {
    float s, sm, half, inv, up;     // the scale; the scale, its half, reciprocal and factor as worked on
};

// amax_bits: the bits of the row's largest magnitude (as unsigned numbers, those
// of an infinity or NaN are the largest of all).
__device__ __forceinline__ CodeScale code_scale(uint32_t amax_bits) {
    CodeScale c;
    if (amax_bits >= 0x7f800000u) {
        c.s = __uint_as_float(0x7fffffffu);
        c.sm = c.half = c.inv = 0.0f;
        c.up = 1.0f;
        return c;
    }
    c.s = __fdiv_rn(__uint_as_float(amax_bits), 127.0f);
    c.up = c.s < 7.88860905e-31f ? 1.2676506e30f : 1.0f;       // 2^-100, 2^100
    c.sm = __fmul_rn(c.s, c.up);
    c.half = 0.5f * c.sm;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(c.inv) : "f"(c.sm));     // a first guess is all it gives
    if (c.s == 0.0f) c.inv = 0.0f;
    return c;
}

// The code of x, given its first guess q.
__device__ __forceinline__ float code_settle(float x, float q, const CodeScale& c) {
    const float r = __fmaf_rn(-q, c.sm, x);
    if (r > c.half || (r == c.half && x > 0.0f)) q += 1.0f;
    else if (r < -c.half || (r == -c.half && x < 0.0f)) q -= 1.0f;
    return q;
}

__device__ __forceinline__ int code_of(float x, const CodeScale& c) {
    if (c.inv == 0.0f) return 0;        // zero or non-finite rows (uniform over the row)
    x = __fmul_rn(x, c.up);
    return (int)fminf(fmaxf(code_settle(x, rintf(__fmul_rn(x, c.inv)), c), -127.0f), 127.0f);
}

// Eight codes as two words.  Adding 1.5 * 2^23 rounds x * inv to a whole number
// whose two's complement is the sum's low byte; the remainders' magnitudes are
// compared with half a scale all eight at once, and only eight that have one at
// or past it are settled one by one.  (bf16 rows have such border cases: half of
// a row's largest value is 63.5 scales, and about one value in a thousand is it.)
// PLAIN: the row's scale is a normal one (plain_scale).
__device__ __forceinline__ bool plain_scale(const CodeScale& c) { return c.up == 1.0f && c.inv != 0.0f; }

template <bool PLAIN>
__device__ __forceinline__ uint2 codes8(const f32x2 (&v)[4], const CodeScale& c) {
    uint32_t b[8];
    if constexpr (PLAIN) {
        const f32x2 magic = pair(12582912.0f, 12582912.0f), inv = pair(c.inv, c.inv), sm = pair(c.sm, c.sm);
        float worst = 0.0f;
        f32x2 r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x2 t = fma2(v[j], inv, magic);
            const float2 h = halves(t);
            b[2 * j] = __float_as_uint(h.x);
            b[2 * j + 1] = __float_as_uint(h.y);
            r[j] = fma2(sub2(magic, t), sm, v[j]);      // v - q * s
            const float2 e = halves(r[j]);
            worst = max_abs3(worst, e.x, e.y);
        }
        if (worst >= c.half) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = j & 1 ? halves(v[j >> 1]).y : halves(v[j >> 1]).x;
                const float e = j & 1 ? halves(r[j >> 1]).y : halves(r[j >> 1]).x;
                const float away = __uint_as_float(__float_as_uint(e) ^ (__float_as_uint(x) & 0x80000000u));
                const uint32_t one = x < 0.0f ? ~0u : 1u;
                if (away >= c.half) b[j] += one;
                else if (away < -c.half) b[j] -= one;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = (uint32_t)code_of(j & 1 ? halves(v[j >> 1]).y : halves(v[j >> 1]).x, c);
    }
    return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
}

__device__ __forceinline__ void pairs8(const float (&v)[8], f32x2 (&p)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = pair(v[2 * j], v[2 * j + 1]);
}

// Reductions over the threads of a row (blockDim.x, up to 16 warps; a CTA has
// blockDim.y rows at a time), every thread getting the result, in a fixed order.
// Two sets of 16 words are used in turn, so that one barrier a reduction is
// enough; words of absent warps are zero.
constexpr int kRowGroups = 8;           // most rows of a CTA at a time

// GROUPS: blockDim.y may be above 1, and each row has a named barrier of its own.
// (A barrier named at run time makes a CTA hold all sixteen, of which an SM has 64:
// kernels without groups use the CTA's.)
template <bool GROUPS>
struct RowReduce {
    uint32_t (*red)[16];
    int turn;
    __device__ __forceinline__ RowReduce(uint32_t (*r)[16]) : red(r + (GROUPS ? 2 * threadIdx.y : 0)), turn(0) {
        if (threadIdx.x < 32) red[threadIdx.x >> 4][threadIdx.x & 15] = 0;
        __syncthreads();
    }
    __device__ __forceinline__ const uint4* exchange(uint32_t v) {
        uint32_t* r = red[turn];
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
        if (GROUPS) asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(blockDim.x) : "memory");
        else __syncthreads();
        return reinterpret_cast<const uint4*>(r);
    }
    __device__ __forceinline__ float sum(float v) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (blockDim.x == 32) return v;
        const uint4* r = exchange(__float_as_uint(v));
        float s = 0.0f;
        for (int i = 0; i < (int)blockDim.x; i += 128) {
            const uint4 w = r[i >> 7];
            s += (__uint_as_float(w.x) + __uint_as_float(w.y)) + (__uint_as_float(w.z) + __uint_as_float(w.w));
        }
        return s;
    }
    __device__ __forceinline__ uint32_t max(uint32_t v) {
        v = __reduce_max_sync(0xffffffffu, v);
        if (blockDim.x == 32) return v;
        const uint4* r = exchange(v);
        uint32_t m = 0;
        for (int i = 0; i < (int)blockDim.x; i += 128) {
            const uint4 w = r[i >> 7];
            m = ::max(m, ::max(::max(w.x, w.y), ::max(w.z, w.w)));
        }
        return m;
    }
};

// Where a thread's values of a row lie, chunk by chunk of eight.  VEC: its chunk
// i is elements 8 c .. 8 c + 7 with c = i * threads + its number; else value j of
// it is element (8 i + j) * threads + its number, so that a warp's single-element
// accesses are neighbours.  Past the row's end values count as 0 and nothing is
// written.
template <bool VEC>
__device__ __forceinline__ int elem(int i, int j) {
    return VEC ? 8 * (i * (int)blockDim.x + (int)threadIdx.x) + j : (8 * i + j) * (int)blockDim.x + (int)threadIdx.x;
}

// Eight values of a row as they are stored (a whole VEC chunk of 16-bit values in
// the first four words), and those as fp32.  Apart, so that the loads of several
// rows can be in flight before the first is converted.
struct Raw8 {
    uint32_t r[8];
};

template <bool VEC>
__device__ __forceinline__ void load_raw(const void* p, int type, int64_t row0, int i, int cols, Raw8& raw) {
    if (VEC && elem<VEC>(i, 0) + 8 <= cols) {
        const char* q = reinterpret_cast<const char*>(p) + (row0 + elem<VEC>(i, 0)) * (type == ELQ_F32 ? 4 : 2);
        const uint4 a = reinterpret_cast<const uint4*>(q)[0];
        raw.r[0] = a.x; raw.r[1] = a.y; raw.r[2] = a.z; raw.r[3] = a.w;
        if (type == ELQ_F32) {
            const uint4 b = reinterpret_cast<const uint4*>(q)[1];
            raw.r[4] = b.x; raw.r[5] = b.y; raw.r[6] = b.z; raw.r[7] = b.w;
        }
        return;
    }
    if (type == ELQ_F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            raw.r[j] = elem<VEC>(i, j) < cols ? reinterpret_cast<const uint32_t*>(p)[row0 + elem<VEC>(i, j)] : 0;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            raw.r[j] = elem<VEC>(i, j) < cols ? reinterpret_cast<const uint16_t*>(p)[row0 + elem<VEC>(i, j)] : 0;
    }
}

template <bool VEC>
__device__ __forceinline__ void raw_values(const Raw8& raw, int type, int i, int cols, float (&v)[8]) {
    if (type == ELQ_F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(raw.r[j]);
    } else if (VEC && elem<VEC>(i, 0) + 8 <= cols) {
        widen8(make_uint4(raw.r[0], raw.r[1], raw.r[2], raw.r[3]), type, v);
    } else if (type == ELQ_BF16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = bf16_lo(raw.r[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __half2float(__ushort_as_half((unsigned short)raw.r[j]));
    }
}

template <bool VEC>
__device__ __forceinline__ void get8(const void* p, int type, int64_t row0, int i, int cols, float (&v)[8]) {
    Raw8 raw;
    load_raw<VEC>(p, type, row0, i, cols, raw);
    raw_values<VEC>(raw, type, i, cols, v);
}

template <bool VEC>
__device__ __forceinline__ void put8(void* p, int type, int64_t row0, int i, int cols, const float (&v)[8]) {
    if (VEC && elem<VEC>(i, 0) + 8 <= cols) {
        store8(p, type, row0 + elem<VEC>(i, 0), v);
        return;
    }
    if (type == ELQ_F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (elem<VEC>(i, j) < cols) reinterpret_cast<float*>(p)[row0 + elem<VEC>(i, j)] = v[j];
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const uint32_t w = type == ELQ_BF16 ? pack_bf16(v[j], v[j + 1]) : pack_f16(v[j], v[j + 1]);
        uint16_t* d = reinterpret_cast<uint16_t*>(p) + row0;
        if (elem<VEC>(i, j) < cols) d[elem<VEC>(i, j)] = (uint16_t)w;
        if (elem<VEC>(i, j + 1) < cols) d[elem<VEC>(i, j + 1)] = (uint16_t)(w >> 16);
    }
}

template <bool VEC>
__device__ __forceinline__ void put_codes8(int8_t* q, int64_t row0, int i, int cols, const float (&v)[8],
                                           const CodeScale& cs) {
    if (VEC && elem<VEC>(i, 0) + 8 <= cols) {
        f32x2 p[4];
        pairs8(v, p);
        *reinterpret_cast<uint2*>(q + row0 + elem<VEC>(i, 0)) = plain_scale(cs) ? codes8<true>(p, cs) : codes8<false>(p, cs);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = elem<VEC>(i, j);
        if (e < cols) q[row0 + e] = (int8_t)code_of(v[j], cs);
    }
}

// The largest of m and the values' magnitudes, a NaN if there is one.
__device__ __forceinline__ float amax8(float m, const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) m = max_abs3(m, v[j], v[j + 1]);
    return m;
}
__device__ __forceinline__ float amax8(float m, const f32x2 (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max_abs3(m, halves(v[j]).x, halves(v[j]).y);
    return m;
}

__device__ __forceinline__ float sumsq8(float s, const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s = __fmaf_rn(v[j], v[j], s);
    return s;
}

// 1 / sqrt(mean + eps), by the reciprocal of the length and rsqrtf (2 ulp): the
// row's factor within four roundings beside the sum's own.
__device__ __forceinline__ float rstd_of(float ss, float inv_cols, float eps) {
    return rsqrtf(__fmaf_rn(ss, inv_cols, eps));
}

// A row's factor from its threads' sums of squares.  Where their sum passes fp32 (values from
// 1.8e19 / sqrt(cols) on) it is taken again after `down`, which has multiplied the values by 2^-80;
// the factor is then that of those.  The sum is the same for all threads of the row, and so is the way.
constexpr float kDown = 8.27180613e-25f;        // 2^-80

// COMPACT: one copy of the code for both, a loop, which is what kernels short of registers want
// (777 x 1283 fp16 residual norm: 8.6 us, 11.2 without); the others do without the loop (2048 x 4096
// bf16: 18.1 us, 18.3 with).
template <bool COMPACT, typename Reduce, typename Sum, typename Down>
__device__ __forceinline__ float row_rstd(Reduce& rr, float inv_cols, float eps, Sum sum, Down down) {
    const float inf = __uint_as_float(0x7f800000u), low = __fmul_rn(__fmul_rn(eps, kDown), kDown);
    if constexpr (COMPACT) {
        float e = eps;
#pragma unroll 1
        while (true) {
            const float ss = rr.sum(sum());
            if (ss != inf || e != eps) return rstd_of(ss, inv_cols, e);
            down();
            e = low;
        }
    } else {
        const float ss = rr.sum(sum());
        if (ss != inf) return rstd_of(ss, inv_cols, eps);
        down();
        return rstd_of(rr.sum(sum()), inv_cols, low);
    }
}

// silu(g) * u in the formula's own steps: expf (CUDA's, within one ulp, 2^-23 of its value), the
// sum, the quotient and the product.  The quotient is Markstein's: q = g / d by an approximate
// reciprocal (2^-23), then its remainder added back once, which leaves 2^-45 beside the one
// rounding.  So h is within 5 * 2^-24 of its value.  Where d passes 2^126 (g < -87.3) the
// reciprocal is flushed and h is zero; the bound on -g keeps d finite there.  (By __fdiv_rn the
// same values came at 28 us for 16384 x 2048, against 19.7.)
__device__ __forceinline__ f32x2 swiglu2(f32x2 g, f32x2 u) {
    const float2 a = halves(g);
    const f32x2 z = pair(-a.x, -a.y);
    const float dx = __fadd_rn(1.0f, expf(fminf(-a.x, 88.0f))), dy = __fadd_rn(1.0f, expf(fminf(-a.y, 88.0f)));
    float rx, ry;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rx) : "f"(-dx));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ry) : "f"(-dy));
    const f32x2 r = pair(rx, ry), q = mul2(z, r);              // -1 / d, g / d
    return mul2(fma2(fma2(q, pair(dx, dy), z), r, q), u);       // q * d - g is minus the remainder
}

// The eight source values of chunk ci of output row `row` (the quantisers'
// inputs before quantising, or the x of a norm).  B: rows of a combine in flight.
template <int OP, bool VEC, int B>
__device__ __forceinline__ void source8(const RowArgs& a, int64_t row, int64_t src, int ci, float (&v)[8]) {
    if (OP == ROW_QUANT) {
        if (src < 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        } else {
            get8<VEC>(a.x, a.x_type, src * a.ldx, ci, a.cols, v);
        }
    } else if (OP == ROW_SWIGLU) {
        float u[8];
        Raw8 rg, ru;
        load_raw<VEC>(a.x, a.x_type, row * a.ldx, ci, a.cols, rg);
        load_raw<VEC>(a.x, a.x_type, row * a.ldx + a.cols, ci, a.cols, ru);
        raw_values<VEC>(rg, a.x_type, ci, a.cols, v);
        raw_values<VEC>(ru, a.x_type, ci, a.cols, u);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float2 h = halves(swiglu2(pair(v[j], v[j + 1]), pair(u[j], u[j + 1])));
            v[j] = h.x;
            v[j + 1] = h.y;
        }
    } else if (OP == ROW_COMBINE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        // B rows at a time: all their positions, then all their pieces, in flight together
        for (int i0 = 0; i0 < a.k; i0 += B) {
            float w[B];
            int64_t p[B];
            Raw8 raw[B];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                p[i] = i0 + i < a.k ? a.index[row * a.k + i0 + i] : -1;
                w[i] = i0 + i < a.k ? a.weights[row * a.k + i0 + i] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < B; ++i)
                if (p[i] >= 0 && p[i] < a.x_rows) load_raw<VEC>(a.x, a.x_type, p[i] * a.ldx, ci, a.cols, raw[i]);
#pragma unroll
            for (int i = 0; i < B; ++i) {
                if (p[i] < 0 || p[i] >= a.x_rows) continue;
                float o[8];
                raw_values<VEC>(raw[i], a.x_type, ci, a.cols, o);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __fmaf_rn(w[i], o[j], v[j]);
            }
        }
    } else {
        get8<VEC>(a.x, a.x_type, row * a.ldx, ci, a.cols, v);
    }
}

template <int NV>
__device__ __forceinline__ float sumsq(const float (&v)[NV][8]) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) s = sumsq8(s, v[i]);
    return s;
}
template <int NV>
__device__ __forceinline__ void times(float (&v)[NV][8], float f) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = __fmul_rn(v[i][j], f);
}

template <bool VEC>
__device__ __forceinline__ void weight8(const float* w, int i, int cols, float (&v)[8]) {
    if (w) {
        get8<VEC>(w, ELQ_F32, 0, i, cols, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 1.0f;
    }
}

__device__ __forceinline__ float residual1(float y, float rstd, float w, float g, float res_scale, float h) {
    return __fmaf_rn(g, __fmul_rn(__fmul_rn(y, rstd), w), __fmul_rn(res_scale, h));
}

// The gate's values of chunk i.
template <bool VEC>
__device__ __forceinline__ void gate8(const RowArgs& a, int64_t row, int i, float (&g)[8]) {
    const float* gr = a.gate ? a.gate + (row / a.gate_rows) * a.gate_ld : nullptr;
    if (gr && a.gate_cols == 1) {
        const float g0 = gr[0];
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = g0;
    } else {
        weight8<VEC>(gr, i, a.cols, g);
    }
}

// v (y's values) -> h' = res_scale * h + gate * (y * rstd * w); 0 past the end.
template <bool VEC>
__device__ __forceinline__ void residual8(const RowArgs& a, int i, float rstd, const float (&w)[8], const float (&g)[8],
                                          const float (&h)[8], float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float r = residual1(v[j], rstd, w[j], g[j], a.res_scale, h[j]);
        v[j] = elem<VEC>(i, j) < a.cols ? r : 0.0f;
    }
}

// v -> v * rstd * w, the normalised row.
__device__ __forceinline__ void norm8(const float (&w)[8], float rstd, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(__fmul_rn(v[j], rstd), w[j]);
}

// VPT: chunks a thread holds in registers (VPT * blockDim.x >= ceil(cols / 8)),
// or 0: none, every step reads its inputs again.  With one chunk a thread the row
// kernels are short of warps, not of registers: 56 leave 1152 threads an SM.
template <int OP, int VPT, bool VEC>
__global__ void __maxnreg__(VPT == 1 && OP != ROW_COMBINE ? 56 : 128) k_rows(const __grid_constant__ RowArgs a) {
    __shared__ __align__(16) uint32_t red[2][16];
    pdl_trigger();
    RowReduce<false> rr(red);
    const int nch = (int)((a.cols + 8ll * blockDim.x - 1) / (8ll * blockDim.x));      // chunks of a thread
    constexpr int NV = VPT > 0 ? VPT : 1, B = VPT == 1 ? 8 : VPT == 2 ? 4 : 2;
    const bool codes = a.n_type == ELQ_I8;
    int8_t* q = reinterpret_cast<int8_t*>(a.n);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        int64_t src = row;
        if (OP == ROW_QUANT && a.index) {
            const int64_t i = a.index[row];
            src = i < 0 || i / a.div >= a.x_rows ? -1 : i / a.div;
        }
        float v[NV][8];
        if constexpr (VPT > 0) {
            constexpr bool NORM = OP == ROW_RMS || OP == ROW_RESIDUAL;
            const float* w_last = OP == ROW_RMS ? a.w : a.w_next;
            // One chunk a thread: the weights too are fetched before the first reduction.
            constexpr bool EARLY = VPT == 1;
            float h[OP == ROW_RESIDUAL ? NV : 1][8], w[8], g[8], wn[8];
            if constexpr (EARLY && OP == ROW_RESIDUAL) {
                weight8<VEC>(a.w, 0, a.cols, w);
                gate8<VEC>(a, row, 0, g);
            }
            if constexpr (EARLY && NORM) weight8<VEC>(w_last, 0, a.cols, wn);
            if constexpr (OP == ROW_RESIDUAL) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {      // past the last chunk these are zeros
                    Raw8 ry, rh;
                    load_raw<VEC>(a.x, a.x_type, row * a.ldx, i, a.cols, ry);
                    load_raw<VEC>(a.h, a.h_type, row * a.ldh, i, a.cols, rh);
                    raw_values<VEC>(ry, a.x_type, i, a.cols, v[i]);
                    raw_values<VEC>(rh, a.h_type, i, a.cols, h[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
                    if (i < nch) source8<OP, VEC, B>(a, row, src, i, v[i]);
                }
            }
            if constexpr (OP == ROW_RESIDUAL) {
                const float rstd = row_rstd<true>(rr, a.inv_cols, a.eps, [&] { return sumsq(v); }, [&] { times(v, kDown); });
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (i >= nch) continue;
                    if constexpr (!EARLY) {
                        weight8<VEC>(a.w, i, a.cols, w);
                        gate8<VEC>(a, row, i, g);
                    }
                    residual8<VEC>(a, i, rstd, w, g, h[i], v[i]);
                    put8<VEC>(a.h_out, a.h_type, row * a.ld_out, i, a.cols, v[i]);
                }
                if (!a.n) continue;
            }
            if constexpr (NORM) {
                const float rstd = row_rstd<true>(rr, a.inv_cols, a.eps, [&] { return sumsq(v); }, [&] { times(v, kDown); });
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (i >= nch) continue;
                    if constexpr (!EARLY) weight8<VEC>(w_last, i, a.cols, wn);
                    norm8(wn, rstd, v[i]);
                    if (!codes) put8<VEC>(a.n, a.n_type, row * a.ldn, i, a.cols, v[i]);
                }
                if (!codes) continue;
            }
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) m = amax8(m, v[i]);
            const CodeScale cs = code_scale(rr.max(__float_as_uint(m)));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i < nch) put_codes8<VEC>(q, row * a.ldn, i, a.cols, v[i], cs);
            }
            if (threadIdx.x == 0) a.scale[row] = cs.s;
        } else {
            float(&t)[8] = v[0];
            float rstd = 0.0f, rstd2 = 0.0f;
            // the row's values at chunk i: source, then the residual update,
            // as far as the statistics so far allow
            auto value = [&](int i) {
                source8<OP, VEC, B>(a, row, src, i, t);
                if constexpr (OP == ROW_RESIDUAL) {
                    float h[8], w[8], g[8];
                    get8<VEC>(a.h, a.h_type, row * a.ldh, i, a.cols, h);
                    weight8<VEC>(a.w, i, a.cols, w);
                    gate8<VEC>(a, row, i, g);
                    residual8<VEC>(a, i, rstd, w, g, h, t);
                }
            };
            auto normed = [&](int i) {
                float w[8];
                weight8<VEC>(OP == ROW_RMS ? a.w : a.w_next, i, a.cols, w);
                norm8(w, rstd2, t);
            };
            // the factor of the values that `get` puts into t, which are read again each time
            auto factor = [&](auto&& get) {
                float f = 1.0f;
                auto sum = [&] {
                    float ss = 0.0f;
                    for (int i = 0; i < nch; ++i) {
                        get(i);
                        times(v, f);
                        ss = sumsq8(ss, t);
                    }
                    return ss;
                };
                const float r = row_rstd<true>(rr, a.inv_cols, a.eps, sum, [&] { f = kDown; });
                return __fmul_rn(r, f);
            };
            if constexpr (OP == ROW_RESIDUAL)
                rstd = factor([&](int i) { source8<OP, VEC, B>(a, row, src, i, t); });
            if (OP == ROW_RMS || (OP == ROW_RESIDUAL && a.n)) rstd2 = factor(value);
            CodeScale cs = code_scale(0);
            if (codes && a.n) {
                float m = 0.0f;
                for (int i = 0; i < nch; ++i) {
                    value(i);
                    if (OP == ROW_RMS || OP == ROW_RESIDUAL) normed(i);
                    m = amax8(m, t);
                }
                cs = code_scale(rr.max(__float_as_uint(m)));
                if (threadIdx.x == 0) a.scale[row] = cs.s;
            }
            // h_out may be h and n may be x: each element's inputs are read
            // here before its outputs are written, by the same thread
            for (int i = 0; i < nch; ++i) {
                value(i);
                if (OP == ROW_RESIDUAL) put8<VEC>(a.h_out, a.h_type, row * a.ld_out, i, a.cols, t);
                if (OP == ROW_RMS || (OP == ROW_RESIDUAL && a.n)) normed(i);
                if (!a.n) continue;
                if (codes) put_codes8<VEC>(q, row * a.ldn, i, a.cols, t, cs);
                else put8<VEC>(a.n, a.n_type, row * a.ldn, i, a.cols, t);
            }
        }
    }
}

// ---- rows through shared memory ---------------------------------------------------
//
// What a row costs besides its values' arithmetic is kept small, since the codes'
// rounding alone is some ten instructions a value and the SMs have about 30 to
// give per value at HBM speed: a thread's pieces lie at fixed byte offsets (from
// a row's start and in shared memory), their valid parts are worked out once, and
// the copies' zero fill stands in for bounds checks when they are read back.

// 16 bytes to shared memory, asynchronously; of the source only `bytes` are read
// and the rest is zero.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}

__device__ __forceinline__ void lds_pairs(uint32_t a, f32x2& x, f32x2& y) {
    asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(a));
}

// The pieces of a row, in order: x's (SwiGLU: the gate's, then the up's), h's,
// a gate that changes from row to row; and of the weights: the written norm's, and
// the product of the post-norm's and a gate that all rows share.  Every fp32 chunk
// of eight has two pieces, others one.
inline __host__ __device__ constexpr int planes_of(int type) { return type == ELQ_F32 ? 2 : 1; }

template <int VPT>
struct Lane {
    int nv[VPT];                // values of this thread's chunks
    uint32_t first;             // shared-memory address of its first piece
    int row_bytes16;            // bytes between its chunks at 16 bits a value: 16 * threads, also between pieces

    // its chunks of a row at `src` into pieces from `at` on; `on` 0: zeros
    __device__ __forceinline__ void fetch(uint32_t at, const uint8_t* src, int type, int on) const {
        if (type == ELQ_F32) {
            src += threadIdx.x * 32;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                copy16(at + (2 * i) * row_bytes16, src + (int64_t)(2 * i) * row_bytes16, on * 4 * min(nv[i], 4));
                copy16(at + (2 * i + 1) * row_bytes16, src + (int64_t)(2 * i) * row_bytes16 + 16,
                       on * 4 * max(nv[i] - 4, 0));
            }
        } else {
            src += threadIdx.x * 16;
#pragma unroll
            for (int i = 0; i < VPT; ++i) copy16(at + i * row_bytes16, src + (int64_t)i * row_bytes16, on * 2 * nv[i]);
        }
    }
    __device__ __forceinline__ void read(uint32_t at, int i, int type, f32x2 (&v)[4]) const {
        if (type == ELQ_F32) {
            lds_pairs(at + (2 * i) * row_bytes16, v[0], v[1]);
            lds_pairs(at + (2 * i + 1) * row_bytes16, v[2], v[3]);
        } else {
            float w[8];
            widen8(lds16(at + i * row_bytes16), type, w);
            pairs8(w, v);
        }
    }
    // v to a row at dst (its first value), rounded to type
    __device__ __forceinline__ void write(uint8_t* dst, int i, int type, const f32x2 (&p)[4]) const {
        const float v[8] = {halves(p[0]).x, halves(p[0]).y, halves(p[1]).x, halves(p[1]).y,
                            halves(p[2]).x, halves(p[2]).y, halves(p[3]).x, halves(p[3]).y};
        if (nv[i] == 8) {
            if (type == ELQ_F32) store8(dst + threadIdx.x * 32 + (int64_t)(2 * i) * row_bytes16, type, 0, v);
            else store8(dst + threadIdx.x * 16 + (int64_t)i * row_bytes16, type, 0, v);
        } else {
            const int e0 = 8 * threadIdx.x + i * (row_bytes16 >> 1);
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < nv[i]) store1(dst, type, e0 + j, v[j]);
        }
    }
    template <bool PLAIN>
    __device__ __forceinline__ void write_codes(int8_t* dst, int i, const f32x2 (&v)[4], const CodeScale& cs) const {
        const int e0 = 8 * threadIdx.x + i * (row_bytes16 >> 1);
        const uint2 w = codes8<PLAIN>(v, cs);
        if (nv[i] == 8) {
            *reinterpret_cast<uint2*>(dst + e0) = w;
        } else {
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < nv[i]) dst[e0 + j] = (int8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
        }
    }
};

// The sum of squares of a thread's values.
template <int VPT>
__device__ __forceinline__ float sumsq(const f32x2 (&v)[VPT][4]) {
    f32x2 s = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fma2(v[i][j], v[i][j], s);
    const float2 h = halves(s);
    return __fadd_rn(h.x, h.y);
}
template <int VPT>
__device__ __forceinline__ void times(f32x2 (&v)[VPT][4], float f) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = mul2(v[i][j], pair(f, f));
}

// A CTA works on blockDim.y rows at a time, blockDim.x threads each, which share
// the weights in shared memory.  D stages: the rows in shared memory per row
// worked on, D - 1 of them on their way.  XT: x's type (a residual norm's: of h and n too), or
// 0xff: as the arguments say.
constexpr int kAnyType = 0xff;
constexpr int kPipeThreads4 = 384;     // most threads with four chunks each

template <int OP, int VPT, int D, int XT>
__global__ void __launch_bounds__(VPT == 1 ? kRowThreads : kPipeThreads4, 2) k_pipe(const __grid_constant__ RowArgs a) {
    extern __shared__ uint4 sm[];
    __shared__ __align__(16) uint32_t red[2 * kRowGroups][16];
    const int T = blockDim.x, xt = XT == kAnyType ? a.x_type : XT, ht = OP == ROW_RESIDUAL && XT != kAnyType ? XT : a.h_type, nt = OP == ROW_RESIDUAL && XT != kAnyType ? XT : a.n_type;
    Lane<VPT> ln;
    ln.row_bytes16 = 16 * T;
    ln.first = (uint32_t)__cvta_generic_to_shared(sm) + 16 * threadIdx.x;
#pragma unroll
    for (int i = 0; i < VPT; ++i) ln.nv[i] = min(8, max(0, a.cols - 8 * ((int)threadIdx.x + i * T)));
    const bool codes = nt == ELQ_I8;
    const bool gate_all = OP == ROW_RESIDUAL && a.gate && a.gate_cols > 1 && a.gate_rows >= a.rows;
    const bool gate_row = OP == ROW_RESIDUAL && a.gate && a.gate_cols > 1 && a.gate_rows < a.rows;
    const int plane = VPT * 16 * T;         // bytes of one piece of all the CTA's chunks
    const int stage_bytes = a.row_planes * plane;
    const uint32_t ring = ln.first + a.w_planes * plane + threadIdx.y * D * stage_bytes;
    const int ox = planes_of(xt) * plane, oh = ox, og = ox + planes_of(ht) * plane;
    const int64_t bx = a.ldx * (xt == ELQ_F32 ? 4 : 2), bh = a.ldh * (ht == ELQ_F32 ? 4 : 2);
    const int64_t bo = a.ld_out * (ht == ELQ_F32 ? 4 : 2), bn = a.ldn * (codes ? 1 : nt == ELQ_F32 ? 4 : 2);
    const uint8_t* x = reinterpret_cast<const uint8_t*>(a.x);
    const uint8_t* hp = reinterpret_cast<const uint8_t*>(a.h);
    uint8_t* op = reinterpret_cast<uint8_t*>(a.h_out);
    uint8_t* np = reinterpret_cast<uint8_t*>(a.n);

    // the source row of an output row: -1 a gathered row that is not there, -2 past the end
    auto source = [&](int64_t row) -> int64_t {
        if (row >= a.rows) return -2;
        if (OP != ROW_QUANT || !a.index) return row;
        const int i = a.index[row];
        return i < 0 || i / a.div >= a.x_rows ? -1 : i / a.div;
    };
    auto fetch = [&](uint32_t at, int64_t row, int64_t src) {
        if (src != -2) {
            const uint8_t* p = x + (src < 0 ? 0 : src) * bx;
            ln.fetch(at, p, xt, OP != ROW_QUANT || src >= 0);
            if (OP == ROW_SWIGLU) ln.fetch(at + ox, p + (int64_t)a.cols * (xt == ELQ_F32 ? 4 : 2), xt, 1);
            if (OP == ROW_RESIDUAL) ln.fetch(at + oh, hp + src * bh, ht, 1);
            if (gate_row)
                ln.fetch(at + og, reinterpret_cast<const uint8_t*>(a.gate + (row / a.gate_rows) * a.gate_ld), ELQ_F32, 1);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    pdl_trigger();
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    const float* w_last = OP == ROW_RMS ? a.w : a.n ? a.w_next : nullptr;     // of the norm that is written
    const uint32_t w_first = ln.first + 2 * plane;                              // w * gate, where either is given
    const bool wg = OP == ROW_RESIDUAL && (a.w || gate_all);
    if (threadIdx.y == 0 && w_last)         // joins the first row's group
        ln.fetch(ln.first, reinterpret_cast<const uint8_t*>(w_last), ELQ_F32, 1);
#pragma unroll
    for (int j = 0; j < D - 1; ++j) fetch(ring + j * stage_bytes, row + j * step, source(row + j * step));
    int64_t ahead = source(row + (D - 1) * step);
    if (wg && threadIdx.y == 0) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float w[8], g[8];
            weight8<true>(a.w, i, a.cols, w);
            weight8<true>(gate_all ? a.gate : nullptr, i, a.cols, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __fmul_rn(w[j], g[j]);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(w_first + (2 * i + j) * ln.row_bytes16),
                             "f"(w[4 * j]), "f"(w[4 * j + 1]), "f"(w[4 * j + 2]), "f"(w[4 * j + 3])
                             : "memory");
        }
    }
    if ((OP == ROW_RMS || OP == ROW_RESIDUAL) && blockDim.y > 1)        // the other rows' threads read the weights too
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    RowReduce<OP == ROW_RMS || OP == ROW_RESIDUAL> rr(red);             // a barrier of the CTA

    for (int st = 0; row < a.rows; row += step, st = st + 1 == D ? 0 : st + 1) {
        fetch(ring + (st == 0 ? D - 1 : st - 1) * stage_bytes, row + (D - 1) * step, ahead);
        ahead = source(row + D * step);
        asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
        const uint32_t at = ring + st * stage_bytes;
        f32x2 v[VPT][4];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            ln.read(at, i, xt, v[i]);
            if (OP == ROW_SWIGLU) {
                f32x2 u[4];
                ln.read(at + ox, i, xt, u);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = swiglu2(v[i][j], u[j]);
            }
        }
        if constexpr (OP == ROW_RESIDUAL) {
            const float rstd = row_rstd<false>(rr, a.inv_cols, a.eps, [&] { return sumsq(v); }, [&] { times(v, kDown); });
            const float g0 = a.gate && a.gate_cols == 1 ? a.gate[(row / a.gate_rows) * a.gate_ld] : 1.0f;
            uint8_t* o = op + row * bo;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                f32x2 h[4], w[4];
                // past the row's end y and h are 0, and so is h'
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = mul2(v[i][j], pair(rstd, rstd));
                if (wg) {
                    ln.read(w_first, i, ELQ_F32, w);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i][j] = mul2(v[i][j], w[j]);
                }
                ln.read(at + oh, i, ht, h);
#pragma unroll
                for (int j = 0; j < 4; ++j) h[j] = mul2(pair(a.res_scale, a.res_scale), h[j]);
                if (gate_row) {
                    ln.read(at + og, i, ELQ_F32, w);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i][j] = fma2(w[j], v[i][j], h[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i][j] = fma2(pair(g0, g0), v[i][j], h[j]);
                }
                ln.write(o, i, ht, v[i]);
            }
            if (!a.n) continue;
        }
        if constexpr (OP == ROW_RMS || OP == ROW_RESIDUAL) {
            const float rstd = row_rstd<false>(rr, a.inv_cols, a.eps, [&] { return sumsq(v); }, [&] { times(v, kDown); });
            uint8_t* o = np + row * bn;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = mul2(v[i][j], pair(rstd, rstd));
                if (w_last) {
                    f32x2 w[4];
                    ln.read(ln.first, i, ELQ_F32, w);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i][j] = mul2(v[i][j], w[j]);
                }
                if (!codes) ln.write(o, i, nt, v[i]);
            }
            if (!codes) continue;
        }
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) m = amax8(m, v[i]);
        const CodeScale cs = code_scale(rr.max(__float_as_uint(m)));
        int8_t* q = reinterpret_cast<int8_t*>(np) + row * bn;
        if (plain_scale(cs)) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) ln.template write_codes<true>(q, i, v[i], cs);
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i) ln.template write_codes<false>(q, i, v[i], cs);
        }
        if (threadIdx.x == 0) a.scale[row] = cs.s;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

}  // namespace elqops
