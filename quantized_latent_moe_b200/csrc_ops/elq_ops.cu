// elq_ops.cu -- the C ABI declared in include/elq_ops.h: host-side validation,
// the choice of kernel, tensor maps and launches.  No allocation, no
// synchronisation (except elq_ops_status, which is documented as blocking).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "../../include/elq_ops.h"
#include "ops_mma.cuh"

using namespace elqops;

namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxK = 65536;            // 65536 * 128 * 128 = 2^30: the int32 sum cannot overflow
constexpr int kMaxExperts = 1024;
constexpr int kMaxSize = 1 << 30;       // rows, channels or columns: their sums with a tile stay below 2^31

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline elq_status status_of(cudaError_t e) { return e == cudaSuccess ? ELQ_OK : ELQ_ERR_CUDA; }
inline bool float_type(int32_t t) { return t == ELQ_F32 || t == ELQ_BF16 || t == ELQ_F16; }
inline int type_bytes(int32_t t) { return t == ELQ_F32 ? 4 : t == ELQ_I8 ? 1 : 2; }

int device_sms() {
    static int cache[kMaxDevices] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
    if (!cache[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
        cache[dev] = n;
    }
    return cache[dev];
}

// A product (early) may start while the row kernel before it drains: it sets itself
// up, and waits for that kernel's completion before it touches global memory.  Only
// this edge is programmatic.  Row kernels are launched plainly, so that no CTA of
// theirs ever waits on an SM, and products let nothing start before their end: with
// both, a chain of row kernels and products stopped for good (row CTAs that waited
// for a product shared its SMs while its CTAs still allocated TMEM and waited for
// their cluster).
template <typename Args>
cudaError_t launch(void (*kern)(Args), dim3 grid, dim3 threads, size_t smem, cudaStream_t s, const Args& a, bool early,
                   int cluster = 1) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (early) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

// ---- row kernels -----------------------------------------------------------------

constexpr int kPipeSmem = 200 * 1024;       // most shared memory of a k_pipe CTA

template <int OP, int VPT, int D, int XT>
cudaError_t launch_pipe_t(const RowArgs& a, int threads, int groups, size_t smem, cudaStream_t s) {
    static bool optin[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices || !optin[dev]) {
        e = cudaFuncSetAttribute(k_pipe<OP, VPT, D, XT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPipeSmem);
        // all of the SM's memory as shared memory: by itself the driver gave four CTAs' worth
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k_pipe<OP, VPT, D, XT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) optin[dev] = true;
    }
    // as many CTAs as fit, by registers (64 a thread with one chunk, 80 with more) and by shared memory
    const int fit = std::max(1, std::min((VPT == 1 ? 1024 : 768) / (threads * groups), (int)(224 * 1024 / (smem + 2048))));
    const dim3 grid((unsigned)std::min<int64_t>((a.rows + groups - 1) / groups, (int64_t)device_sms() * fit));
    return launch(k_pipe<OP, VPT, D, XT>, grid, dim3(threads, groups), smem, s, a, false);
}

// Rows through shared memory; false where they are too long for it.
template <int OP>
bool launch_pipe(RowArgs a, cudaStream_t s, cudaError_t* e) {
    const int chunks = (a.cols + 7) / 8;
    if (chunks > 4 * kPipeThreads4) return false;
    // Few rows: one chunk a thread, the shortest way through a row.  Many: up to
    // four, since a thread's work per row besides its values (reductions, the
    // scale, addresses) is as much as two or three chunks'.
    const bool many = a.rows > 2 * device_sms();
    int vpt = chunks <= kRowThreads ? 1 : 4;
    if (many && chunks > 32) vpt = 4;
    const int threads = std::max(32, ((chunks + vpt - 1) / vpt + 31) / 32 * 32);
    const bool gate = OP == ROW_RESIDUAL && a.gate && a.gate_cols > 1;
    a.w_planes = OP == ROW_RMS ? 2 : OP == ROW_RESIDUAL ? 4 : 0;
    a.row_planes = planes_of(a.x_type) * (OP == ROW_SWIGLU ? 2 : 1) + (OP == ROW_RESIDUAL ? planes_of(a.h_type) : 0) +
                   (gate && a.gate_rows < a.rows ? 2 : 0);
    const size_t plane = (size_t)vpt * threads * 16;
    // Many rows with weights to share: several rows of a CTA at a time (2048 x 4096
    // bf16, residual norm: 18.1 us with three, 22.8 with one; norm: 12.2 and 19.0).
    int groups = 1, d = 1;
    auto smem = [&](int g, int dd) { return (a.w_planes + (size_t)g * dd * a.row_planes) * plane; };
    if (many) {
        if (vpt == 4 && a.w_planes)
            groups = std::min(kRowGroups, kPipeThreads4 / threads);
        // three stages a row, else two, and fewer rows before fewer stages
        while (groups > 1 && smem(groups, 2) > kPipeSmem) --groups;
        d = smem(groups, 3) <= kPipeSmem ? 3 : smem(groups, 2) <= kPipeSmem ? 2 : 1;
    }
    if (smem(groups, d) > kPipeSmem) return false;
    auto go = [&](auto v, auto dd) {
        constexpr int V = decltype(v)::value, D = decltype(dd)::value;
        if constexpr (OP == ROW_RESIDUAL) {
            // one 16-bit type throughout is known at compile time (2048 x 4096 bf16: 18.1 us, 22.0 with
            // the types chosen as it runs); mixed types are not
            const bool same = a.x_type == a.h_type && a.n && a.n_type == a.h_type;
            if (same && a.x_type == ELQ_BF16) *e = launch_pipe_t<OP, V, D, ELQ_BF16>(a, threads, groups, smem(groups, d), s);
            else if (same && a.x_type == ELQ_F16) *e = launch_pipe_t<OP, V, D, ELQ_F16>(a, threads, groups, smem(groups, d), s);
            else *e = launch_pipe_t<OP, V, D, kAnyType>(a, threads, groups, smem(groups, d), s);
        } else if (a.x_type == ELQ_F32) *e = launch_pipe_t<OP, V, D, ELQ_F32>(a, threads, groups, smem(groups, d), s);
        else if (a.x_type == ELQ_BF16) *e = launch_pipe_t<OP, V, D, ELQ_BF16>(a, threads, groups, smem(groups, d), s);
        else *e = launch_pipe_t<OP, V, D, ELQ_F16>(a, threads, groups, smem(groups, d), s);
    };
    using one = std::integral_constant<int, 1>;
    using two = std::integral_constant<int, 2>;
    using three = std::integral_constant<int, 3>;
    using four = std::integral_constant<int, 4>;
    if (vpt == 1) d == 1 ? go(one(), one()) : go(one(), three());
    else d == 1 ? go(four(), one()) : d == 2 ? go(four(), two()) : go(four(), three());
    return true;
}

template <int OP, int VPT, bool VEC>
cudaError_t launch_rows_t(const RowArgs& a, int threads, cudaStream_t s) {
    const int64_t most = (int64_t)device_sms() * std::max(1, 2048 / threads);
    return launch(k_rows<OP, VPT, VEC>, dim3((unsigned)std::min<int64_t>(a.rows, most)), threads, 0, s, a, false);
}

// k_rows: chunks of a row in registers, as few a thread as 512 threads allow, or none (every step
// reads its inputs again) for rows past 16384 values.  Aligned rows come here where k_pipe does not
// take them (from 12289 values on, fp32 residual norms with a gate a row from 10241).  Of those the
// quantiser and the plain norm read again, with half the registers and more warps an SM (2048 x
// 14336 bf16: 39 and 42 us, 54 and 62 from registers); SwiGLU and the residual norm, which would do
// their arithmetic again too, keep them (73 us, 103 read again; 1024 rows 59 us, 86).
template <int OP, bool VEC>
cudaError_t launch_rows_v(const RowArgs& a, cudaStream_t s) {
    const int chunks = (a.cols + 7) / 8;
    const int vpt = chunks <= kRowThreads ? 1 : chunks <= 2 * kRowThreads ? 2 : chunks <= 4 * kRowThreads ? 4 : 0;
    const int threads = vpt == 0 ? kRowThreads : std::max(32, ((chunks + vpt - 1) / vpt + 31) / 32 * 32);
    if constexpr (OP == ROW_COMBINE || !VEC) {      // aligned rows of the others, this short, go through k_pipe
        if (vpt == 1) return launch_rows_t<OP, 1, VEC>(a, threads, s);
        if (vpt == 2) return launch_rows_t<OP, 2, VEC>(a, threads, s);
    }
    if constexpr (!VEC || (OP != ROW_QUANT && OP != ROW_RMS)) {
        if (vpt == 4) return launch_rows_t<OP, 4, VEC>(a, threads, s);
    }
    return launch_rows_t<OP, 0, VEC>(a, kRowThreads, s);
}

// Whether rows `ld` elements of type t apart keep 16-byte alignment.
inline bool wide(const void* p, int64_t ld, int32_t t) {
    return !p || (aligned(p, 16) && (ld * type_bytes(t)) % 16 == 0);
}

template <int OP>
elq_status launch_rows(RowArgs a, void* stream) {
    a.inv_cols = 1.0f / (float)a.cols;
    bool vec = wide(a.x, a.ldx, a.x_type) && wide(a.h, a.ldh, a.h_type) && wide(a.h_out, a.ld_out, a.h_type) &&
               wide(a.n, a.ldn, a.n_type) && wide(a.w, 0, ELQ_F32) && wide(a.w_next, 0, ELQ_F32);
    if (a.gate && a.gate_cols > 1) vec = vec && wide(a.gate, a.gate_ld, ELQ_F32);
    if (OP == ROW_SWIGLU) vec = vec && a.cols % 8 == 0;     // the up half starts on a vector
    cudaStream_t s = (cudaStream_t)stream;
    if constexpr (OP != ROW_COMBINE) {
        cudaError_t e = cudaSuccess;
        if (vec && launch_pipe<OP>(a, s, &e)) return status_of(e);
    }
    return status_of(vec ? launch_rows_v<OP, true>(a, s) : launch_rows_v<OP, false>(a, s));
}

// The codes a row call writes.
elq_status check_codes(const int8_t* q, int64_t ldq, const float* scale, int64_t rows, int32_t cols) {
    if (ldq < cols) return ELQ_ERR_INVALID_ARG;
    if (ldq % 16) return ELQ_ERR_ALIGNMENT;
    if (rows == 0) return ELQ_OK;
    if (!q || !scale) return ELQ_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(scale, 4)) return ELQ_ERR_ALIGNMENT;
    return ELQ_OK;
}

// ---- products --------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, []() {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

bool encode(CUtensorMap* m, int es, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = map_encoder();
    if (!fn) return false;
    const cuuint32_t one[3] = {1, 1, 1};
    return fn(m, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, rank,
              const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Product {
    const void* x;
    int64_t ldx;                // elements
    const float* sx;
    int M;
    const void* w;
    int64_t ldw, w_stride;
    const float *sw, *bias;
    int E, N, K;
    const int32_t* offsets;
    void* y;
    int y_type;
    int64_t ldy;
    int kind;
    int stall = 0;              // a test's (MmaArgs)
    uint64_t wait_ns = kOpsWaitNs;
};

template <int KIND, int R, int U>
cudaError_t launch_gemv(const Product& p, cudaStream_t s) {
    const int es = KIND == KIND_I8 ? 1 : 2;
    GemvArgs a;
    a.x = (const uint8_t*)p.x;
    a.ldx = p.ldx * es;
    a.sx = p.sx;
    a.w = (const uint8_t*)p.w;
    a.ldw = p.ldw * es;
    a.w_stride = p.w_stride * es;
    a.sw = p.sw;
    a.bias = p.bias;
    a.M = p.M;
    a.E = p.E;
    a.N = p.N;
    a.Kb = p.K * es;
    a.offsets = p.offsets;
    a.y = p.y;
    a.y_type = p.y_type;
    a.ldy = p.ldy;
    const int per = kGemvWarps * R;
    // four CTAs an SM, each going on to further channels: what a CTA does before its
    // first weights arrive (finding its group) is done once for all of them
    const int groups = p.offsets ? std::min(p.E, p.M) : 1;
    const int most = std::max(1, 4 * device_sms() / groups);
    const dim3 grid((unsigned)std::min<int64_t>(most, ((int64_t)p.N + per - 1) / per), groups);
    return launch(k_gemv<KIND, R, U>, grid, 32 * kGemvWarps, 0, s, a, true);
}

// Channels a warp takes at a time (R) and pieces of each in flight (U).  8-bit
// codes: four channels, two pieces, where that leaves work for every warp (8 rows
// of 8 experts of 2048 x 1792: 7.8 us, 9.0 with two and four; tensor cores 9.2);
// else two and four (1 row 4096 -> 1792: 4.4 us, 5.3 with four and two).  16-bit:
// two and four, since each weight is widened into registers.
cudaError_t launch_gemv(const Product& p, cudaStream_t s) {
    if (p.kind == KIND_BF16) return launch_gemv<KIND_BF16, 2, 4>(p, s);
    if (p.kind == KIND_F16) return launch_gemv<KIND_F16, 2, 4>(p, s);
    const int64_t channels = (int64_t)p.N * (p.offsets ? std::min(p.E, p.M) : 1);
    return channels >= 40 * device_sms() ? launch_gemv<KIND_I8, 4, 2>(p, s) : launch_gemv<KIND_I8, 2, 4>(p, s);
}

// Row tiles, in whole copied boxes of 32 rows a CTA: as many rows as the group can have up to 256; a dense product takes
// the tile that needs the fewest steps: waves of tiles, each as long as its MMAs
// (or, below 128 rows, as its weight tile takes to arrive).
int row_tile(const Product& p, int sms, int cg) {
    const int step = 32 * cg;
    int bn = std::min(256, (p.M + step - 1) / step * step);
    if (p.offsets || p.M <= 64) return bn;
    const int64_t ch_tiles = ((int64_t)p.N + cg * kTileCh - 1) / (cg * kTileCh);
    int64_t best = INT64_MAX;
    for (int t = bn; t >= 64; t -= step) {
        const int64_t tiles = (p.M + t - 1) / t * ch_tiles, at_once = sms / cg;
        const int64_t cost = (tiles + at_once - 1) / at_once * (std::max(t, 128) + 16);
        if (cost < best) {
            best = cost;
            bn = t;
        }
    }
    return bn;
}

// The arguments that the tensor-core kernels share, but for the tile and ring.
template <int KIND>
bool mma_args(const Product& p, int cg, MmaArgs& a) {
    const int es = KIND == KIND_I8 ? 1 : 2;
    const cuuint64_t dw[3] = {(cuuint64_t)p.K, (cuuint64_t)p.N, (cuuint64_t)p.E};
    const cuuint64_t sw[2] = {(cuuint64_t)(p.ldw * es), (cuuint64_t)((p.E > 1 ? p.w_stride : p.ldw * p.N) * es)};
    const cuuint32_t bw[3] = {(cuuint32_t)(kStepBytes / es), kTileCh, 1};
    const cuuint64_t dx[2] = {(cuuint64_t)p.K, (cuuint64_t)p.M};
    const cuuint64_t sx[1] = {(cuuint64_t)(p.ldx * es)};
    const cuuint32_t bx[2] = {(cuuint32_t)(kStepBytes / es), kBoxRows};
    a.offsets = p.offsets;
    a.M = p.M;
    a.E = p.E;
    a.N = p.N;
    a.Kb = p.K * es;
    a.split = 1;
    a.stall = p.stall;
    a.wait_ns = p.wait_ns;
    a.idesc = mma_idesc(KIND, cg);
    a.sx = p.sx;
    a.sw = p.sw;
    a.bias = p.bias;
    a.y = p.y;
    a.y_type = p.y_type;
    a.ldy = p.ldy;
    return encode(&a.tw, es, 3, p.w, dw, sw, bw) && encode(&a.tx, es, 2, p.x, dx, sx, bx);
}

// Large shared memory for a kernel, once per device.  The tensor-core kernels take
// all of an SM's: TMEM is allocated by an instruction that blocks while another CTA
// of the SM holds it, and CTAs of a cluster wait for one another, so that two such
// kernels on two streams, sharing SMs, could wait in a circle.
template <typename K>
bool mma_optin(K kern, bool* done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev >= 0 && dev < kMaxDevices && done[dev]) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMmaSmemMax) != cudaSuccess) return false;
    if (dev >= 0 && dev < kMaxDevices) done[dev] = true;
    return true;
}

template <int KIND, int CG>
elq_status launch_mma(const Product& p, cudaStream_t s) {
    static bool optin[kMaxDevices];
    const int sms = device_sms() / CG * CG;
    const int64_t ch_tiles = ((int64_t)p.N + CG * kTileCh - 1) / (CG * kTileCh);
    MmaArgs a;
    if (!mma_args<KIND>(p, CG, a) || !mma_optin(k_mma<KIND, CG>, optin)) return ELQ_ERR_CUDA;
    a.bn = row_tile(p, sms, CG);
    const int64_t units = ((int64_t)p.M / a.bn + p.E + 1) * ch_tiles;
    if (units > INT32_MAX) return ELQ_ERR_UNSUPPORTED;
    const int hdr = kMmaHdr + 2 * (p.E + 1) * 4 + 1024, stage = kABytes + a.bn / CG * kStepBytes;
    a.stages = std::min(kMmaStagesMax, (kMmaSmemMax - hdr) / stage);
    const dim3 grid((unsigned)std::min<int64_t>(sms, units * CG));
    return status_of(launch(k_mma<KIND, CG>, grid, kMmaThreads, kMmaSmemMax, s, a, true, CG));
}

// CTAs per tile and rows of a tile for a dense product split over K; 1 where no
// split is quicker.  In nanoseconds, as measured: a K step of a lone tile of bn
// rows takes 150 + 0.4 bn, the exchange 400 + 17 a row.  (4096 -> 1792: 16 rows
// 6.6 us against 10.4 unsplit, 256 rows 9.0 against 12.5; from about 1000 rows on
// the tiles fill the SMs.)
int split_plan(const Product& p, int* bn) {
    const int sms = device_sms(), steps = (p.K + kStepBytes - 1) / kStepBytes;
    const int64_t ch_tiles = ((int64_t)p.N + kTileCh - 1) / kTileCh;
    const int bn1 = row_tile(p, sms, 1);
    if ((p.M + bn1 - 1) / bn1 * ch_tiles > sms) return 1;
    int best = 1;
    int64_t cost = (int64_t)steps * (150 + bn1 * 2 / 5);
    for (int t = 32; t <= 256 && t < p.M + 32; t += 32) {
        const int64_t tiles = (p.M + t - 1) / t * ch_tiles;
        for (int split = 2; split <= 8 && split <= steps && tiles * split <= sms; split *= 2) {
            const int64_t c = (int64_t)((steps + split - 1) / split) * (150 + t * 2 / 5) + 400 + 17 * std::min(t, p.M);
            if (c < cost) {
                cost = c;
                best = split;
                *bn = t;
            }
        }
    }
    return best;
}

elq_status launch_split(const Product& p, int split, int bn, cudaStream_t s) {
    static bool optin[kMaxDevices];
    MmaArgs a;
    if (!mma_args<KIND_I8>(p, 1, a) || !mma_optin(k_split, optin)) return ELQ_ERR_CUDA;
    const int stage = kABytes + bn * kStepBytes, hdr = 512 + 1024;
    const int steps = (int)((a.Kb + kStepBytes - 1) / kStepBytes), share = (steps + split - 1) / split;
    a.bn = bn;
    a.split = split;
    a.stages = std::min({kMmaStagesMax, (kMmaSmemMax - hdr) / stage, share});
    const int64_t tiles = (p.M + bn - 1) / bn * (((int64_t)p.N + kTileCh - 1) / kTileCh);
    return status_of(launch(k_split, dim3((unsigned)(tiles * split)), kMmaThreads, kMmaSmemMax, s, a, true, split));
}

// Pairs of CTAs where their tiles (an expert with rows has one at least) fill the
// SMs more than once: they bring the rows to shared memory half as often (8192 x
// 4096 x 4096 codes: 87.6 us against 99.6; 16384 rows over 128 experts: 96.6 against
// 108.4).  Where one wave has them all, single CTAs spread over more SMs (2048 x
// 1792 x 4096: 16.7 against 18.2).
template <int KIND>
elq_status launch_mma(const Product& p, cudaStream_t s) {
    if constexpr (KIND == KIND_I8) {        // dense products are of codes
        int bn = 0;
        const int split = p.offsets ? 1 : split_plan(p, &bn);
        if (split > 1) return launch_split(p, split, bn, s);
    }
    const int64_t pairs = ((int64_t)p.N + 2 * kTileCh - 1) / (2 * kTileCh);
    const int64_t row_tiles = std::max<int64_t>(std::min(p.E, p.M), (p.M + 255) / 256);
    return pairs * row_tiles > device_sms() / 2 ? launch_mma<KIND, 2>(p, s) : launch_mma<KIND, 1>(p, s);
}

// The register GEMV for grouped products of up to 8 rows (above, the tensor cores
// read the weights faster: 16 rows of 16 experts); dense ones of up to 4, or 8 of a
// matrix below 256 KB (4096 -> 1792: 4.3 us for one row, 6.1 for four, 8.9 for six,
// against 5.2 split over K; 512 -> 512, six rows: 1.9 against 3.1).
bool few_rows(const Product& p) {
    if (p.offsets || p.M <= 4) return p.M <= 8;
    return p.M <= 8 && (int64_t)p.N * p.K <= 1 << 18;
}

elq_status run_product(const Product& p, cudaStream_t s) {
    if (few_rows(p)) return status_of(launch_gemv(p, s));
    return p.kind == KIND_I8 ? launch_mma<KIND_I8>(p, s) : p.kind == KIND_BF16 ? launch_mma<KIND_BF16>(p, s)
                                                                               : launch_mma<KIND_F16>(p, s);
}

elq_status check_i8_matmul(const Product& p, int64_t T) {
    if (T < 0 || p.N < 1 || p.K < 1 || p.ldx < p.K || p.ldw < p.K || p.ldy < p.N) return ELQ_ERR_INVALID_ARG;
    if (!float_type(p.y_type) || p.K > kMaxK || T > kMaxSize || p.N > kMaxSize) return ELQ_ERR_UNSUPPORTED;
    if (p.ldx % 16 || p.ldw % 16) return ELQ_ERR_ALIGNMENT;
    if (T == 0) return ELQ_OK;
    if (!p.x || !p.sx || !p.w || !p.sw || !p.y) return ELQ_ERR_INVALID_ARG;
    if (!aligned(p.x, 16) || !aligned(p.w, 16) || !aligned(p.y, 16) || !aligned(p.sx, 4) || !aligned(p.sw, 4) ||
        !aligned(p.bias, 4))
        return ELQ_ERR_ALIGNMENT;
    return ELQ_OK;
}

}  // namespace

extern "C" {

elq_status elq_quantize_i8(const void* x, int32_t x_type, int64_t x_rows, int32_t cols, int64_t ldx,
                           const int32_t* index, int32_t div, int64_t rows, int8_t* q, int64_t ldq, float* scale,
                           void* stream) {
    if (rows < 0 || x_rows < 0 || cols < 1 || ldx < cols || div < 1) return ELQ_ERR_INVALID_ARG;
    if (!index && rows > 0 && (div != 1 || rows > x_rows)) return ELQ_ERR_INVALID_ARG;
    if (!float_type(x_type) || cols > kMaxSize) return ELQ_ERR_UNSUPPORTED;
    const elq_status st = check_codes(q, ldq, scale, rows, cols);
    if (st != ELQ_OK || rows == 0) return st;
    if (!x || x_rows == 0) return ELQ_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(index, 4)) return ELQ_ERR_ALIGNMENT;
    RowArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rows = rows;
    a.cols = cols;
    a.x = x;
    a.x_type = x_type;
    a.ldx = ldx;
    a.x_rows = x_rows;
    a.index = index;
    a.div = div;
    a.n = q;
    a.n_type = ELQ_I8;
    a.ldn = ldq;
    a.scale = scale;
    return launch_rows<ROW_QUANT>(a, stream);
}

elq_status elq_swiglu_i8(const void* gu, int32_t x_type, int64_t rows, int32_t I, int64_t ld, int8_t* q, int64_t ldq,
                         float* scale, void* stream) {
    if (rows < 0 || I < 1 || ld < 2ll * I) return ELQ_ERR_INVALID_ARG;
    if (!float_type(x_type) || I > kMaxSize) return ELQ_ERR_UNSUPPORTED;
    const elq_status st = check_codes(q, ldq, scale, rows, I);
    if (st != ELQ_OK || rows == 0) return st;
    if (!gu) return ELQ_ERR_INVALID_ARG;
    if (!aligned(gu, 16)) return ELQ_ERR_ALIGNMENT;
    RowArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rows = rows;
    a.cols = I;
    a.x = gu;
    a.x_type = x_type;
    a.ldx = ld;
    a.n = q;
    a.n_type = ELQ_I8;
    a.ldn = ldq;
    a.scale = scale;
    return launch_rows<ROW_SWIGLU>(a, stream);
}

elq_status elq_combine_i8(const void* o, int32_t o_type, int64_t o_rows, int32_t cols, int64_t ldo, const int32_t* pos,
                          const float* weights, int64_t T, int32_t k, int8_t* q, int64_t ldq, float* scale,
                          void* stream) {
    if (T < 0 || o_rows < 0 || cols < 1 || ldo < cols || k < 1 || k > 64) return ELQ_ERR_INVALID_ARG;
    if (!float_type(o_type) || cols > kMaxSize) return ELQ_ERR_UNSUPPORTED;
    const elq_status st = check_codes(q, ldq, scale, T, cols);
    if (st != ELQ_OK || T == 0) return st;
    if (!o || o_rows == 0 || !pos || !weights) return ELQ_ERR_INVALID_ARG;
    if (!aligned(o, 16) || !aligned(pos, 4) || !aligned(weights, 4)) return ELQ_ERR_ALIGNMENT;
    RowArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rows = T;
    a.cols = cols;
    a.x = o;
    a.x_type = o_type;
    a.ldx = ldo;
    a.x_rows = o_rows;
    a.index = pos;
    a.weights = weights;
    a.k = k;
    a.n = q;
    a.n_type = ELQ_I8;
    a.ldn = ldq;
    a.scale = scale;
    return launch_rows<ROW_COMBINE>(a, stream);
}

elq_status elq_i8_matmul(const int8_t* x, int64_t ldx, const float* sx, int64_t T, const int8_t* w, int64_t ldw,
                         const float* sw, const float* bias, int32_t N, int32_t K, void* y, int32_t y_type, int64_t ldy,
                         void* stream) {
    const Product p = {x, ldx, sx, (int)T, w, ldw, 0, sw, bias, 1, N, K, nullptr, y, y_type, ldy, KIND_I8};
    const elq_status st = check_i8_matmul(p, T);
    return st != ELQ_OK || T == 0 ? st : run_product(p, (cudaStream_t)stream);
}

elq_status elq_test_i8_matmul_timeout(const int8_t* x, int64_t ldx, const float* sx, int64_t T, const int8_t* w,
                                      int64_t ldw, const float* sw, int32_t N, int32_t K, float* y, int64_t ldy,
                                      int32_t stall, uint64_t budget_ns, void* stream) {
    Product p = {x, ldx, sx, (int)T, w, ldw, 0, sw, nullptr, 1, N, K, nullptr, y, ELQ_F32, ldy, KIND_I8};
    const elq_status st = check_i8_matmul(p, T);
    if (st != ELQ_OK) return st;
    if (stall < 1 || stall > 2 || budget_ns < 1000000ull || budget_ns > kOpsWaitNs) return ELQ_ERR_INVALID_ARG;
    if (T == 0 || few_rows(p)) return ELQ_ERR_UNSUPPORTED;
    p.stall = stall;
    p.wait_ns = budget_ns;
    return run_product(p, (cudaStream_t)stream);
}

elq_status elq_grouped_matmul(const void* x, int32_t x_type, int64_t ldx, const float* sx, int64_t M, const void* w,
                              int64_t ldw, int64_t w_stride, const float* sw, int32_t E, int32_t N, int32_t K,
                              const int32_t* offsets, void* y, int32_t y_type, int64_t ldy, void* stream) {
    if (M < 0 || E < 1 || N < 1 || K < 1 || ldx < K || ldw < K || ldy < N) return ELQ_ERR_INVALID_ARG;
    if (E > 1 && w_stride < (int64_t)(N - 1) * ldw + K) return ELQ_ERR_INVALID_ARG;
    if (x_type != ELQ_I8 && x_type != ELQ_BF16 && x_type != ELQ_F16) return ELQ_ERR_UNSUPPORTED;
    if (!float_type(y_type) || (x_type != ELQ_I8 && y_type != ELQ_F32 && y_type != x_type)) return ELQ_ERR_UNSUPPORTED;
    if (K > kMaxK || E > kMaxExperts || M > kMaxSize || N > kMaxSize) return ELQ_ERR_UNSUPPORTED;
    const int es = type_bytes(x_type);
    if ((ldx * es) % 16 || (ldw * es) % 16 || (E > 1 && (w_stride * es) % 16)) return ELQ_ERR_ALIGNMENT;
    if (M == 0) return ELQ_OK;
    if (!x || !w || !offsets || !y) return ELQ_ERR_INVALID_ARG;
    if ((x_type == ELQ_I8) != (sx != nullptr) || (x_type == ELQ_I8) != (sw != nullptr)) return ELQ_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(sx, 4) || !aligned(sw, 4) ||
        !aligned(offsets, 4))
        return ELQ_ERR_ALIGNMENT;
    const Product p = {x, ldx, sx, (int)M, w, ldw, w_stride, sw, nullptr, E, N, K, offsets, y, y_type, ldy,
                       x_type == ELQ_I8 ? KIND_I8 : x_type == ELQ_BF16 ? KIND_BF16 : KIND_F16};
    return run_product(p, (cudaStream_t)stream);
}

elq_status elq_rms_norm(const void* x, int32_t x_type, int64_t T, int32_t cols, int64_t ldx, const float* weight,
                        float eps, void* n, int32_t n_type, int64_t ldn, float* scale, void* stream) {
    if (T < 0 || cols < 1 || ldx < cols || ldn < cols || !(eps > 0.0f) || !std::isfinite(eps))
        return ELQ_ERR_INVALID_ARG;
    if (!float_type(x_type) || (!float_type(n_type) && n_type != ELQ_I8) || cols > kMaxSize)
        return ELQ_ERR_UNSUPPORTED;
    if (n_type == ELQ_I8) {
        const elq_status st = check_codes((const int8_t*)n, ldn, scale, T, cols);
        if (st != ELQ_OK) return st;
    } else if (scale) {
        return ELQ_ERR_INVALID_ARG;
    }
    if (T == 0) return ELQ_OK;
    if (!x || !n) return ELQ_ERR_INVALID_ARG;
    if (n == x && (n_type != x_type || ldn != ldx)) return ELQ_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(n, 16) || !aligned(weight, 4)) return ELQ_ERR_ALIGNMENT;
    RowArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rows = T;
    a.cols = cols;
    a.x = x;
    a.x_type = x_type;
    a.ldx = ldx;
    a.w = weight;
    a.eps = eps;
    a.n = n;
    a.n_type = n_type;
    a.ldn = ldn;
    a.scale = scale;
    return launch_rows<ROW_RMS>(a, stream);
}

elq_status elq_residual_norm(const elq_residual* r, void* stream) {
    if (!r) return ELQ_ERR_INVALID_ARG;
    if (r->T < 0 || r->cols < 1 || r->ldh < r->cols || r->ldy < r->cols || r->ld_out < r->cols)
        return ELQ_ERR_INVALID_ARG;
    if (!(r->eps > 0.0f) || !std::isfinite(r->eps)) return ELQ_ERR_INVALID_ARG;
    if (!float_type(r->h_type) || !float_type(r->y_type) || r->cols > kMaxSize) return ELQ_ERR_UNSUPPORTED;
    const bool next = r->n != nullptr;
    if (next) {
        if (!float_type(r->n_type) && r->n_type != ELQ_I8) return ELQ_ERR_UNSUPPORTED;
        if (r->ldn < r->cols) return ELQ_ERR_INVALID_ARG;
        if (r->n_type == ELQ_I8) {
            const elq_status st = check_codes((const int8_t*)r->n, r->ldn, r->scale, r->T, r->cols);
            if (st != ELQ_OK) return st;
        }
    }
    if (r->scale && !(next && r->n_type == ELQ_I8) && r->T > 0) return ELQ_ERR_INVALID_ARG;
    if (r->gate && (r->gate_rows < 1 || (r->gate_cols != 1 && r->gate_cols != r->cols) || r->gate_ld < r->gate_cols))
        return ELQ_ERR_INVALID_ARG;
    if (r->T == 0) return ELQ_OK;
    if (!r->h || !r->y || !r->h_out) return ELQ_ERR_INVALID_ARG;
    if (r->h_out == r->h && r->ld_out != r->ldh) return ELQ_ERR_INVALID_ARG;
    if (r->h_out == r->y || (next && (r->n == r->h || r->n == r->y || r->n == r->h_out))) return ELQ_ERR_INVALID_ARG;
    if (!aligned(r->h, 16) || !aligned(r->y, 16) || !aligned(r->h_out, 16) || !aligned(r->n, 16) ||
        !aligned(r->post_weight, 4) || !aligned(r->gate, 4) || !aligned(r->next_weight, 4))
        return ELQ_ERR_ALIGNMENT;
    RowArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rows = r->T;
    a.cols = r->cols;
    a.x = r->y;
    a.x_type = r->y_type;
    a.ldx = r->ldy;
    a.h = r->h;
    a.ldh = r->ldh;
    a.h_type = r->h_type;
    a.h_out = r->h_out;
    a.ld_out = r->ld_out;
    a.w = r->post_weight;
    a.gate = r->gate;
    a.gate_rows = r->gate_rows;
    a.gate_ld = r->gate_ld;
    a.gate_cols = r->gate_cols == r->cols ? r->cols : 1;
    a.w_next = r->next_weight;
    a.res_scale = r->res_scale;
    a.eps = r->eps;
    a.n = r->n;
    a.n_type = next ? r->n_type : ELQ_F32;
    a.ldn = r->ldn;
    a.scale = r->scale;
    return launch_rows<ROW_RESIDUAL>(a, stream);
}

elq_status elq_ops_status(void* stream) {
    static std::mutex one;      // g_ops_said is one caller's at a time
    cudaStream_t s = (cudaStream_t)stream;
    if (cudaStreamSynchronize(s) != cudaSuccess) return ELQ_ERR_CUDA;
    int err = 0;
    std::lock_guard<std::mutex> lock(one);
    k_status<<<1, 1, 0, s>>>();
    if (cudaGetLastError() != cudaSuccess ||
        cudaMemcpyFromSymbolAsync(&err, g_ops_said, sizeof(err), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return ELQ_ERR_CUDA;
    return err ? ELQ_ERR_TIMEOUT : ELQ_OK;
}

}  // extern "C"
