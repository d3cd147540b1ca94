// ops_gemv.cuh -- products for a few rows: every weight is read once, straight
// from HBM into registers, and multiplied with up to four rows of activations
// that come from L1.
//
// A warp owns R neighbouring output channels over all of K: lane i takes the
// 16-byte pieces i, i + 32, ... of each channel's row, U of them in flight, and
// the warp's sums meet in a shuffle reduction.  What bounds it is the weights'
// HBM traffic, and for one small matrix the launch and one memory round trip.
// Measured on B200: 1 row 4096 -> 1792 codes 4.3 us, 8 rows of 8 experts of 2048 x
// 1792 7.5 us (3.9 TB/s; bf16 14 us).
#pragma once

#include "ops_rows.cuh"

namespace elqops {

enum Kind { KIND_I8 = 0, KIND_BF16 = 1, KIND_F16 = 2 };

struct GemvArgs {
    const uint8_t* x;           // rows ldx bytes apart
    int64_t ldx;
    const float* sx;
    const uint8_t* w;           // rows ldw bytes apart, experts w_stride
    int64_t ldw, w_stride;
    const float* sw;
    const float* bias;
    int M, E, N, Kb;            // Kb: bytes of a row
    const int32_t* offsets;     // NULL: one group of all M rows
    void* y;
    int y_type;
    int64_t ldy;
};

constexpr int kGemvWarps = 4;

__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// A row's last piece, of n < 16 bytes, read byte by byte; zeros after it.
__device__ __forceinline__ uint4 load_tail(const uint8_t* p, int n) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (i < n) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sums of C values over the warp, by halves: at each step a lane passes on the
// half of its values that its partner keeps.  Lane l ends with the sum of value
// l >> (5 - log2 C).
template <int C, typename T>
__device__ __forceinline__ T warp_sums(T (&v)[C]) {
    const int lane = threadIdx.x & 31;
    int o = 16;
#pragma unroll
    for (int n = C / 2; n >= 1; n >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const T give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
        o >>= 1;
    }
    T s = v[0];
    for (; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

template <int KIND, int R, int TB, typename Acc>
__device__ __forceinline__ void gemv_piece(const uint4 (&w)[R], const uint4 (&x)[TB], Acc (&acc)[R * TB]) {
    if constexpr (KIND == KIND_I8) {
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                int s = acc[r * TB + t];
                s = __dp4a((int)w[r].x, (int)x[t].x, s);
                s = __dp4a((int)w[r].y, (int)x[t].y, s);
                s = __dp4a((int)w[r].z, (int)x[t].z, s);
                acc[r * TB + t] = __dp4a((int)w[r].w, (int)x[t].w, s);
            }
    } else {
        float wf[R][8];
#pragma unroll
        for (int r = 0; r < R; ++r) widen8(w[r], KIND == KIND_BF16 ? ELQ_BF16 : ELQ_F16, wf[r]);
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            float xf[8];
            widen8(x[t], KIND == KIND_BF16 ? ELQ_BF16 : ELQ_F16, xf);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[r * TB + t] = __fmaf_rn(wf[r][j], xf[j], acc[r * TB + t]);
        }
    }
}

// Channels n0 .. n0+R-1 of expert matrix w times rows t0 .. t0+nt-1 (nt <= TB).
template <int KIND, int R, int TB, int U>
__device__ __forceinline__ void gemv_rows(const GemvArgs& a, const uint8_t* w, const float* sw, int n0, int t0, int nt) {
    using Acc = typename std::conditional<KIND == KIND_I8, int, float>::type;
    constexpr int C = R * TB;
    const int lane = threadIdx.x & 31;
    const uint8_t* wr[R];
    const uint8_t* xr[TB];
#pragma unroll
    for (int r = 0; r < R; ++r) wr[r] = w + (int64_t)min(n0 + r, a.N - 1) * a.ldw;
#pragma unroll
    for (int t = 0; t < TB; ++t) xr[t] = a.x + (int64_t)(t0 + min(t, nt - 1)) * a.ldx;
    Acc acc[C];
#pragma unroll
    for (int i = 0; i < C; ++i) acc[i] = 0;
    const int pieces = a.Kb >> 4;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int p0 = lane; p0 < pieces; p0 += 32 * U) {
        uint4 wv[U][R];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r)
                wv[u][r] = p0 + 32 * u < pieces ? ldg_stream(wr[r] + 16 * (int64_t)(p0 + 32 * u)) : zero;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint4 xv[TB];
            if (p0 + 32 * u < pieces) {
#pragma unroll
                for (int t = 0; t < TB; ++t)
                    xv[t] = __ldg(reinterpret_cast<const uint4*>(xr[t] + 16 * (int64_t)(p0 + 32 * u)));
                gemv_piece<KIND, R, TB>(wv[u], xv, acc);
            }
        }
    }
    if ((a.Kb & 15) && lane == 0) {
        uint4 wv[R], xv[TB];
#pragma unroll
        for (int r = 0; r < R; ++r) wv[r] = load_tail(wr[r] + 16 * (int64_t)pieces, a.Kb & 15);
#pragma unroll
        for (int t = 0; t < TB; ++t) xv[t] = load_tail(xr[t] + 16 * (int64_t)pieces, a.Kb & 15);
        gemv_piece<KIND, R, TB>(wv, xv, acc);
    }
    __syncwarp();
    const Acc s = warp_sums<C>(acc);
    constexpr int per = 32 / C;             // lanes that hold each sum
    const int i = lane / per, n = n0 + i / TB, t = i % TB;
    if (lane % per == 0 && n < a.N && t < nt) {
        float v = (float)s;
        if (KIND == KIND_I8) {
            v = __fmul_rn(__fmul_rn(v, __ldg(a.sx + t0 + t)), __ldg(sw + n));
            if (a.bias) v = __fadd_rn(v, __ldg(a.bias + n));
        }
        store1(a.y, a.y_type, (int64_t)(t0 + t) * a.ldy + n, v);
    }
}

__device__ __forceinline__ int clamp_offset(int o, int M) { return min(max(o, 0), M); }

// Offsets clamped to the rows and raised to the largest before them: groups are
// then disjoint whatever the array holds.  One batch of 32 (o: this lane's offset),
// `before` the largest of the batches before, updated.  Warp-collective.
__device__ __forceinline__ int raise_offsets(int o, int M, int& before) {
    o = max(clamp_offset(o, M), before);
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, o, d);
        if (lane >= d) o = max(o, v);
    }
    before = __shfl_sync(0xffffffffu, o, 31);
    return o;
}

// The want-th (from 0) group that has rows: its expert and rows r0 .. r1-1.
// Warp-uniform; false if there is none.
__device__ __forceinline__ bool find_group(const int32_t* offsets, int E, int M, int want, int& e, int& r0, int& r1) {
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int e0 = 0; e0 < E; e0 += 128) {
        int lo[4], hi[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {       // all loads before the scans
            const int i = e0 + 32 * b + lane;
            lo[b] = i < E ? __ldg(offsets + i) : 0;
            hi[b] = i < E ? __ldg(offsets + i + 1) : 0;
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int l0 = raise_offsets(lo[b], M, before);
            const int h0 = max(l0, clamp_offset(hi[b], M));
            uint32_t m = __ballot_sync(0xffffffffu, h0 > l0);
            const int c = __popc(m);
            if (want < c) {
                for (int i = 0; i < want; ++i) m &= m - 1;
                const int l = __ffs(m) - 1;
                e = e0 + 32 * b + l;
                r0 = __shfl_sync(0xffffffffu, l0, l);
                r1 = __shfl_sync(0xffffffffu, h0, l);
                return true;
            }
            want -= c;
        }
    }
    return false;
}

template <int KIND, int R, int U>
__global__ void __launch_bounds__(32 * kGemvWarps) k_gemv(const __grid_constant__ GemvArgs a) {
    pdl_wait();
    int e = 0, r0 = 0, r1 = a.M;        // at most min(E, M) groups have rows, and the grid has that many
    if (a.offsets && !find_group(a.offsets, a.E, a.M, blockIdx.y, e, r0, r1)) return;
    const uint8_t* w = a.w + (int64_t)e * a.w_stride;
    const float* sw = KIND == KIND_I8 ? a.sw + (int64_t)e * a.N : nullptr;
    for (int n0 = (blockIdx.x * kGemvWarps + (threadIdx.x >> 5)) * R; n0 < a.N; n0 += gridDim.x * kGemvWarps * R) {
        for (int t0 = r0; t0 < r1; t0 += 4) {
            const int nt = min(4, r1 - t0);
            if (nt == 1) gemv_rows<KIND, R, 1, U>(a, w, sw, n0, t0, nt);
            else if (nt == 2) gemv_rows<KIND, R, 2, U>(a, w, sw, n0, t0, nt);
            else gemv_rows<KIND, R, 4, U>(a, w, sw, n0, t0, nt);
        }
    }
}

}  // namespace elqops
