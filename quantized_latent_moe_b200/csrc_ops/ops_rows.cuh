// ops_rows.cuh -- the row kernels: activation rows to 8-bit codes (plain,
// gathered, SwiGLU'd, or a weighted sum of expert rows), and the norms before
// and after a block.
//
// All are one pass over memory.  A CTA owns a row at a time (grid-strided): it
// loads the row's inputs once into registers as fp32, takes the row's
// reductions (sum of squares, largest magnitude) by warp shuffles and one
// shared-memory exchange each, and writes the outputs.  What bounds them is
// HBM traffic for many rows and launch-to-finish latency for one.  Rows longer
// than the registers of a CTA hold (16384 values) take the same steps but read
// their inputs again for each step.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/elq_ops.h"

namespace elqops {

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
    float res_scale, eps;
    // outputs
    void* h_out;
    int h_type;
    int64_t ld_out;
    void* n;                    // codes, or the normalised row
    int n_type;
    int64_t ldn;
    float* scale;
};

constexpr int kRowThreads = 512;        // most threads of a CTA
constexpr int kRowMaxCols = kRowThreads * 8 * 4;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ float load1(const void* p, int type, int64_t i) {
    if (type == ELQ_F32) return reinterpret_cast<const float*>(p)[i];
    const uint16_t b = reinterpret_cast<const uint16_t*>(p)[i];
    return type == ELQ_BF16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
}

// Eight consecutive values from element i (a multiple of 8 from a 16-byte
// aligned row).
__device__ __forceinline__ void load8(const void* p, int type, int64_t i, float (&v)[8]) {
    if (type == ELQ_F32) {
        const float4 a = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i)[0];
        const float4 b = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        return;
    }
    const uint4 r = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (type == ELQ_BF16) {
            v[2 * j] = bf16_lo(w[j]);
            v[2 * j + 1] = bf16_hi(w[j]);
        } else {
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

__device__ __forceinline__ uint32_t pack2(int type, float a, float b) {
    if (type == ELQ_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
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
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) =
        make_uint4(pack2(type, v[0], v[1]), pack2(type, v[2], v[3]), pack2(type, v[4], v[5]), pack2(type, v[6], v[7]));
}

// The scale of a row and what its codes need: x / s to the nearest whole
// number, exactly.  rint(|x| * inv) is within one of it; the remainder
// |x| - q * s is exact in fp32 (one fused multiply-add), and its comparison
// with s / 2 settles the rounding, halves away from zero.  A scale below
// 2^-100 is worked on times 2^100 (exact) so that its reciprocal is finite.
struct CodeScale {
    float s, sm, inv, up;       // the scale, the scale and factor it is worked on with
};

// amax_bits: the largest bit pattern of |x| over the row (an infinity or NaN
// has the largest of all).
__device__ __forceinline__ CodeScale code_scale(uint32_t amax_bits) {
    CodeScale c;
    if (amax_bits >= 0x7f800000u) {
        c.s = __uint_as_float(0x7fffffffu);
        c.sm = c.inv = c.up = 0.0f;
        return c;
    }
    c.s = __fdiv_rn(__uint_as_float(amax_bits), 127.0f);
    c.up = c.s < 7.88860905e-31f ? 1.2676506e30f : 1.0f;       // 2^-100, 2^100
    c.sm = __fmul_rn(c.s, c.up);
    c.inv = c.s > 0.0f ? __fdiv_rn(1.0f, c.sm) : 0.0f;
    return c;
}

__device__ __forceinline__ int code_of(float x, const CodeScale& c) {
    if (c.inv == 0.0f) return 0;        // zero or non-finite rows (uniform over the row)
    const float t = __fmul_rn(fabsf(x), c.up);
    float q = rintf(__fmul_rn(t, c.inv));
    const float r2 = 2.0f * __fmaf_rn(-q, c.sm, t);
    if (r2 >= c.sm) q += 1.0f;
    else if (r2 < -c.sm) q -= 1.0f;
    const int i = (int)fminf(q, 127.0f);
    return x < 0.0f ? -i : i;
}

// Reductions over the CTA, every thread getting the result, in a fixed order.
// `red` holds two sets of 32 words used in turn, so that one barrier each is
// enough.
struct RowReduce {
    uint32_t (*red)[32];
    int turn;
    __device__ __forceinline__ float sum(float v) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        const int nw = blockDim.x >> 5;
        if (nw == 1) return v;
        uint32_t* r = red[turn];
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = __float_as_uint(v);
        __syncthreads();
        float s = 0.0f;
        for (int i = 0; i < nw; ++i) s += __uint_as_float(r[i]);
        return s;
    }
    __device__ __forceinline__ uint32_t max(uint32_t v) {
        v = __reduce_max_sync(0xffffffffu, v);
        const int nw = blockDim.x >> 5;
        if (nw == 1) return v;
        uint32_t* r = red[turn];
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
        __syncthreads();
        uint32_t m = 0;
        for (int i = 0; i < nw; ++i) m = ::max(m, r[i]);
        return m;
    }
};

// Where a thread's values of a row lie.  VEC: chunk c of 8 consecutive values
// from element 8 c; else value j of chunk c is element (8 (c / threads) + j) *
// threads + c % threads, so that a warp's single-element accesses are
// neighbours.  Past the row's end values count as 0 and nothing is written.
template <bool VEC>
__device__ __forceinline__ int elem(int c, int j) {
    return VEC ? 8 * c + j : (int)(8 * (c / (int)blockDim.x) + j) * (int)blockDim.x + c % (int)blockDim.x;
}

template <bool VEC>
__device__ __forceinline__ void get8(const void* p, int type, int64_t row0, int c, int cols, float (&v)[8]) {
    if (VEC && 8 * c + 8 <= cols) {
        load8(p, type, row0 + 8 * c, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = elem<VEC>(c, j);
        v[j] = e < cols ? load1(p, type, row0 + e) : 0.0f;
    }
}

template <bool VEC>
__device__ __forceinline__ void put8(void* p, int type, int64_t row0, int c, int cols, const float (&v)[8]) {
    if (VEC && 8 * c + 8 <= cols) {
        store8(p, type, row0 + 8 * c, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = elem<VEC>(c, j);
        if (e < cols) store1(p, type, row0 + e, v[j]);
    }
}

template <bool VEC>
__device__ __forceinline__ void put_codes8(int8_t* q, int64_t row0, int c, int cols, const float (&v)[8],
                                           const CodeScale& cs) {
    if (VEC && 8 * c + 8 <= cols) {
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j >> 2] |= (uint32_t)(code_of(v[j], cs) & 0xff) << (8 * (j & 3));
        *reinterpret_cast<uint2*>(q + row0 + 8 * c) = make_uint2(w[0], w[1]);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = elem<VEC>(c, j);
        if (e < cols) q[row0 + e] = (int8_t)code_of(v[j], cs);
    }
}

__device__ __forceinline__ uint32_t amax8(uint32_t m, const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    return m;
}

__device__ __forceinline__ float sumsq8(float s, const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s = __fmaf_rn(v[j], v[j], s);
    return s;
}

__device__ __forceinline__ float rstd_of(float ss, int cols, float eps) {
    return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)cols), eps)));
}

// The eight source values of chunk c of output row `row` (the quantisers'
// inputs before quantising, or the x of a norm).
template <int OP, bool VEC>
__device__ __forceinline__ void source8(const RowArgs& a, int64_t row, int64_t src, int c, float (&v)[8]) {
    if (OP == ROW_QUANT) {
        if (src < 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        } else {
            get8<VEC>(a.x, a.x_type, src * a.ldx, c, a.cols, v);
        }
    } else if (OP == ROW_SWIGLU) {
        float u[8];
        get8<VEC>(a.x, a.x_type, row * a.ldx, c, a.cols, v);
        get8<VEC>(a.x, a.x_type, row * a.ldx + a.cols, c, a.cols, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // exp(-g) = inf gives g / inf = -0 for a very negative g
            const float e = __expf(-v[j]);
            v[j] = __fmul_rn(__fdiv_rn(v[j], __fadd_rn(1.0f, e)), u[j]);
        }
    } else if (OP == ROW_COMBINE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        for (int i = 0; i < a.k; ++i) {
            const int64_t p = a.index[row * a.k + i];
            if (p < 0 || p >= a.x_rows) continue;
            const float w = a.weights[row * a.k + i];
            float o[8];
            get8<VEC>(a.x, a.x_type, p * a.ldx, c, a.cols, o);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __fmaf_rn(w, o[j], v[j]);
        }
    } else {
        get8<VEC>(a.x, a.x_type, row * a.ldx, c, a.cols, v);
    }
}

template <bool VEC>
__device__ __forceinline__ void weight8(const float* w, int c, int cols, float (&v)[8]) {
    if (w) {
        get8<VEC>(w, ELQ_F32, 0, c, cols, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 1.0f;
    }
}

// v (y's values) -> h' = res_scale * h + gate * (y * rstd * w); 0 past the end.
template <bool VEC>
__device__ __forceinline__ void residual8(const RowArgs& a, int64_t row, int c, float rstd, const float (&h)[8],
                                          float (&v)[8]) {
    float w[8], g[8];
    weight8<VEC>(a.w, c, a.cols, w);
    if (!a.gate) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = 1.0f;
    } else {
        const float* gr = a.gate + (row / a.gate_rows) * a.gate_ld;
        if (a.gate_cols == 1) {
            const float g0 = gr[0];
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = g0;
        } else {
            get8<VEC>(gr, ELQ_F32, 0, c, a.cols, g);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float n = __fmul_rn(__fmul_rn(v[j], rstd), w[j]);
        const float r = __fmaf_rn(g[j], n, __fmul_rn(a.res_scale, h[j]));
        v[j] = elem<VEC>(c, j) < a.cols ? r : 0.0f;
    }
}

// v -> v * rstd * w, the normalised row.
template <bool VEC>
__device__ __forceinline__ void norm8(const float* wt, int c, int cols, float rstd, float (&v)[8]) {
    float w[8];
    weight8<VEC>(wt, c, cols, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(__fmul_rn(v[j], rstd), w[j]);
}

// VPT: chunks a thread holds in registers (VPT * blockDim.x >= ceil(cols / 8)),
// or 0: none, every step reads its inputs again.
template <int OP, int VPT, bool VEC>
__global__ void __launch_bounds__(kRowThreads) k_rows(const __grid_constant__ RowArgs a) {
    __shared__ uint32_t red[2][32];
    RowReduce rr{red, 0};
    const int nch = VEC ? (a.cols + 7) / 8 : (int)blockDim.x * (int)((a.cols + 8ll * blockDim.x - 1) / (8ll * blockDim.x));
    constexpr int NV = VPT > 0 ? VPT : 1;
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
            float h[OP == ROW_RESIDUAL ? NV : 1][8];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
                if (c < nch) source8<OP, VEC>(a, row, src, c, v[i]);
                if constexpr (OP == ROW_RESIDUAL) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
                    if (c < nch) get8<VEC>(a.h, a.h_type, row * a.ldh, c, a.cols, h[i]);
                }
            }
            if constexpr (OP == ROW_RESIDUAL) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i) ss = sumsq8(ss, v[i]);
                const float rstd = rstd_of(rr.sum(ss), a.cols, a.eps);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = threadIdx.x + i * blockDim.x;
                    if (c >= nch) continue;
                    residual8<VEC>(a, row, c, rstd, h[i], v[i]);
                    put8<VEC>(a.h_out, a.h_type, row * a.ld_out, c, a.cols, v[i]);
                }
                if (!a.n) continue;
            }
            if constexpr (OP == ROW_RMS || OP == ROW_RESIDUAL) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i) ss = sumsq8(ss, v[i]);
                const float rstd = rstd_of(rr.sum(ss), a.cols, a.eps);
                const float* wt = OP == ROW_RMS ? a.w : a.w_next;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = threadIdx.x + i * blockDim.x;
                    if (c >= nch) continue;
                    norm8<VEC>(wt, c, a.cols, rstd, v[i]);
                    if (!codes) put8<VEC>(a.n, a.n_type, row * a.ldn, c, a.cols, v[i]);
                }
                if (!codes) continue;
            }
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) m = amax8(m, v[i]);
            const CodeScale cs = code_scale(rr.max(m));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                if (c < nch) put_codes8<VEC>(q, row * a.ldn, c, a.cols, v[i], cs);
            }
            if (threadIdx.x == 0) a.scale[row] = cs.s;
        } else {
            float(&t)[8] = v[0];
            float rstd = 0.0f, rstd2 = 0.0f;
            // the row's values at chunk c: source, then the residual update,
            // as far as the statistics so far allow
            auto value = [&](int c) {
                source8<OP, VEC>(a, row, src, c, t);
                if constexpr (OP == ROW_RESIDUAL) {
                    float h[8];
                    get8<VEC>(a.h, a.h_type, row * a.ldh, c, a.cols, h);
                    residual8<VEC>(a, row, c, rstd, h, t);
                }
            };
            const float* wt = OP == ROW_RMS ? a.w : a.w_next;
            if constexpr (OP == ROW_RESIDUAL) {
                float ss = 0.0f;
                for (int c = threadIdx.x; c < nch; c += blockDim.x) {
                    source8<OP, VEC>(a, row, src, c, t);
                    ss = sumsq8(ss, t);
                }
                rstd = rstd_of(rr.sum(ss), a.cols, a.eps);
            }
            if (OP == ROW_RMS || (OP == ROW_RESIDUAL && a.n)) {
                float ss = 0.0f;
                for (int c = threadIdx.x; c < nch; c += blockDim.x) {
                    value(c);
                    ss = sumsq8(ss, t);
                }
                rstd2 = rstd_of(rr.sum(ss), a.cols, a.eps);
            }
            CodeScale cs = code_scale(0);
            if (codes && a.n) {
                uint32_t m = 0;
                for (int c = threadIdx.x; c < nch; c += blockDim.x) {
                    value(c);
                    if (OP == ROW_RMS || OP == ROW_RESIDUAL) norm8<VEC>(wt, c, a.cols, rstd2, t);
                    m = amax8(m, t);
                }
                cs = code_scale(rr.max(m));
                if (threadIdx.x == 0) a.scale[row] = cs.s;
            }
            // h_out may be h and n may be x: each element's inputs are read
            // here before its outputs are written, by the same thread
            for (int c = threadIdx.x; c < nch; c += blockDim.x) {
                value(c);
                if (OP == ROW_RESIDUAL) put8<VEC>(a.h_out, a.h_type, row * a.ld_out, c, a.cols, t);
                if (OP == ROW_RMS || (OP == ROW_RESIDUAL && a.n)) norm8<VEC>(wt, c, a.cols, rstd2, t);
                if (!a.n) continue;
                if (codes) put_codes8<VEC>(q, row * a.ldn, c, a.cols, t, cs);
                else put8<VEC>(a.n, a.n_type, row * a.ldn, c, a.cols, t);
            }
        }
    }
}

}  // namespace elqops
