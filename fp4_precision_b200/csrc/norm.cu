// norm.cu - RMSNorm of the FP4 layers' bf16 inputs: forward with the
// residual's addition (and the tensor amax or the MXFP4 quantization that the
// next FP4 layer takes), and backward.
//
// Forward, per row of C elements: h = bf16(x + r), rstd = fp32(1 / sqrt(sum
// h^2 / C + eps)), y = bf16(fp32(fp32(h * rstd) * w)). The sum and the root
// are taken in fp64: a bf16 square is exact there, so rstd, y and everything
// quantized from y do not depend on the order of the sum, and the amax and the
// codes are those of qfp4_amax and qfp4_quantize on y bit for bit. The fp64
// work (one conversion and one multiply-add per element) is below a fifth of
// the SM's rate at the speed the rows arrive from HBM.
// Backward: g = dy * w, c = rstd * sum(g h) / C, dx = bf16(rstd * (g - h rstd
// c) + dh), dw = sum over the rows of dy * h * rstd, all in fp32.
//
// Both are bound by HBM: every tensor crosses it once, a row stays in
// registers between the sum and its use. A row belongs to one CTA (C > 1024)
// or one warp; a thread holds 32 elements of it, whole Hadamard groups, so
// that the rotation needs no shuffles. CTAs are persistent: the weight is
// loaded once, and the next row's loads are issued before the row's sum is
// joined. The backward pass of wide rows has them arrive through a ring in
// shared memory.
#include "qfp4_device.cuh"
#include "qfp4_internal.h"

namespace qfp4 {
namespace {

constexpr int kNormElems = 32;        // elements of a row per thread
constexpr int kNormWarpRowC = 1024;   // up to this many columns a row belongs to one warp
constexpr int kNormMaxThreads = 512;  // C <= 16384
constexpr int kNormMaxStages = 4;     // rows in flight per CTA of the backward ring
constexpr int kNormRingBytes = 192 * 1024;

// A thread's 32 elements are NCH chunks of G consecutive ones (G = 16: chunks
// t and t + threads per row; G = 32: chunk t).
template <int G>
struct NormChunks {
    static constexpr int NCH = kNormElems / G;
    int tpr, t;     // threads per row, this thread's index among them
    int chunks;     // chunks in a row
    __device__ __forceinline__ bool has(int i) const { return t + i * tpr < chunks; }
    __device__ __forceinline__ int64_t at(int i) const { return (int64_t)(t + i * tpr) * G; }
    // 16 words of packed bf16 pairs; chunks past the row are zero
    __device__ __forceinline__ void load(const uint16_t* row, uint32_t* w) const {
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int v = 0; v < G / 8; ++v) {
                uint4 q = make_uint4(0, 0, 0, 0);
                if (has(i)) q = *reinterpret_cast<const uint4*>(row + at(i) + 8 * v);
                uint32_t* d = w + i * (G / 2) + 4 * v;
                d[0] = q.x; d[1] = q.y; d[2] = q.z; d[3] = q.w;
            }
    }
    __device__ __forceinline__ void store(uint16_t* row, const uint32_t* w, const void* base, int64_t extent) const {
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int v = 0; v < G / 8; ++v) {
                const uint32_t* s = w + i * (G / 2) + 4 * v;
                if (has(i))
                    *chk(reinterpret_cast<uint4*>(row + at(i) + 8 * v), base, extent) =
                        make_uint4(s[0], s[1], s[2], s[3]);
            }
    }
};

__device__ __forceinline__ uint32_t norm_pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ int64_t rows_extent(int64_t R, int64_t C, int64_t ld) { return R <= 0 ? 0 : ((R - 1) * ld + C) * 2; }

// Sum over the threads of a row, the same in each of them: shuffles, then (a
// row of several warps) one barrier; `red` alternates between two halves, so
// that the next row's partial sums do not overtake this one's.
template <bool WARP_ROW, typename T>
__device__ __forceinline__ T norm_row_sum(T v, T (*red)[kNormMaxThreads / 32], int parity) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (!WARP_ROW) {
        const int warps = blockDim.x >> 5;
        if ((threadIdx.x & 31) == 0) red[parity][threadIdx.x >> 5] = v;
        __syncthreads();
        v = red[parity][0];
        for (int w = 1; w < warps; ++w) v += red[parity][w];
    }
    return v;
}

// NH: -1 no amax, else the Hadamard size of the amax or (QUANT) of the MXFP4
// quantization.
template <int NH, bool QUANT, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? 128 : kNormMaxThreads) rmsnorm_fwd_kernel(const NormParams p) {
    constexpr int G = (QUANT || NH == 32) ? 32 : 16;
    using Chunks = NormChunks<G>;
    __shared__ double red[2][kNormMaxThreads / 32];
    __shared__ float red_max[kNormMaxThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t owners = WARP_ROW ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
    const int64_t first = WARP_ROW ? (int64_t)blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
    const Chunks ch{WARP_ROW ? 32 : (int)blockDim.x, WARP_ROW ? lane : (int)threadIdx.x, (int)(p.C / G)};
    pdl_wait();  // the previous kernel's writes are visible (and its reads done)
    pdl_launch_dependents();

    const int64_t rows_padded = QUANT ? (p.R + 127) / 128 * 128 : p.R;  // scale rows up to the atom are zero
    uint32_t xw[16], rw[16], ww[16];
    ch.load(p.w, ww);
    if (first < p.R) {
        ch.load(p.x + first * p.ldx, xw);
        if (p.res != nullptr) ch.load(p.res + first * p.ldres, rw);
    }
    if (QUANT && blockIdx.x == 0 && threadIdx.x == 0) *chk(p.q_tensor_scale, p.q_tensor_scale, 4) = 1.0f;
    float amax = 0.0f;
    int parity = 0;
    for (int64_t row = first; row < rows_padded; row += owners, parity ^= 1) {
        uint32_t hw[16];
        float rstd = 0.0f;
        if (row < p.R) {
            double ss = 0.0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                hw[i] = p.res != nullptr ? norm_pack(__fadd_rn(bf16lo(xw[i]), bf16lo(rw[i])),
                                                     __fadd_rn(bf16hi(xw[i]), bf16hi(rw[i])))
                                         : xw[i];
                const double a = bf16lo(hw[i]), b = bf16hi(hw[i]);
                ss = __fma_rn(a, a, ss);
                ss = __fma_rn(b, b, ss);
            }
            if (p.h != nullptr) ch.store(p.h + row * p.ldh, hw, p.h, rows_extent(p.R, p.C, p.ldh));
            if (row + owners < p.R) {  // the next row's loads, under this row's sum and outputs
                ch.load(p.x + (row + owners) * p.ldx, xw);
                if (p.res != nullptr) ch.load(p.res + (row + owners) * p.ldres, rw);
            }
            ss = norm_row_sum<WARP_ROW>(ss, red, parity);
            rstd = (float)rsqrt(ss * p.inv_c + p.eps);
            if (ch.t == 0) *chk(p.rstd + row, p.rstd, p.R * 4) = rstd;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                hw[i] = norm_pack(__fmul_rn(__fmul_rn(bf16lo(hw[i]), rstd), bf16lo(ww[i])),
                                  __fmul_rn(__fmul_rn(bf16hi(hw[i]), rstd), bf16hi(ww[i])));
            if (!QUANT || p.y != nullptr) ch.store(p.y + row * p.ldy, hw, p.y, rows_extent(p.R, p.C, p.ldy));
        }
        if constexpr (QUANT) {
            using Grp = Group<kMxfp4, kRtn, NH>;
            static_assert(Grp::G == 32, "32-element MXFP4 blocks");
            uint32_t scode = 0;
            if (row < p.R) {
                const Stream st{0, 0, 0, p.q_round_up};
                ScaleRng srng;
                float v[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    uint32_t x = hw[i];
                    if (NH > 0 && p.signs != 0u) x ^= Grp::sign_mask(p.signs, i);
                    v[2 * i] = bf16lo(x);
                    v[2 * i + 1] = bf16hi(x);
                }
                Grp::rotate(v);
                uint32_t codes[4];
                Grp::quantize(v, 1.0f, nullptr, st, 0, 0, srng, codes, &scode);
                if (ch.has(0))
                    *chk(reinterpret_cast<uint4*>(p.q_codes + row * (p.C / 2) + ch.t * 16), p.q_codes,
                         p.R * (p.C / 2)) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
                else
                    scode = 0;
            }
            // four neighbouring lanes hold the four scales of one word of the atom
            scode |= __shfl_down_sync(0xffffffffu, scode, 1) << 8;
            scode = (scode & 0xFFFFu) | __shfl_down_sync(0xffffffffu, scode, 2) << 16;
            if ((ch.t & 3) == 0 && ch.t < p.q_kb4)
                *chk(reinterpret_cast<uint32_t*>(p.q_scales + ((row / 128) * (p.q_kb4 / 4) + ch.t / 4) * 512 +
                                                 (row % 32) * 16 + ((row / 32) % 4) * 4),
                     p.q_scales, (p.R + 127) / 128 * (p.q_kb4 / 4) * 512) = scode;
        } else if constexpr (NH >= 0) {
            using Grp = Group<kNvfp4, kRtn, NH>;
#pragma unroll
            for (int i = 0; i < Chunks::NCH; ++i) {
                float v[G];
#pragma unroll
                for (int k = 0; k < G / 2; ++k) {
                    uint32_t x = hw[i * (G / 2) + k];
                    if (NH > 0 && p.signs != 0u) x ^= Grp::sign_mask(p.signs, k);
                    v[2 * k] = bf16lo(x);
                    v[2 * k + 1] = bf16hi(x);
                }
                if (ch.has(i)) amax = rot_abs_max<NH, G>(amax, v);
            }
        }
    }
    if constexpr (!QUANT && NH >= 0) {  // the CTA's maximum; c * max |y| = max |c * y|
        if constexpr (NH > 0) amax = __fmul_rn(amax, had_norm<NH>());
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (lane == 0) red_max[warp] = amax;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < (int)(blockDim.x >> 5); ++w) amax = fmaxf(amax, red_max[w]);
            *chk(p.amax_out + blockIdx.x, p.amax_out, (int64_t)gridDim.x * 4) = amax;
        }
    }
}

// ---- backward ------------------------------------------------------------------
// A thread holds up to NV chunks of eight columns (chunks t, t + threads, ...)
// and keeps the weight gradient of its columns in registers over all its rows;
// it leaves once per row owner, as row `owner` of p.dw_partials.
template <int NV>
struct NormBwdThread {
    int t, threads, chunks;
    float dw[8 * NV];
    uint32_t ww[4 * NV];
    __device__ __forceinline__ bool has(int i) const { return t + i * threads < chunks; }
    __device__ __forceinline__ int at(int i) const { return 8 * (t + i * threads); }
    __device__ __forceinline__ void load(const uint16_t* row, uint32_t* w) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint4 q = make_uint4(0, 0, 0, 0);
            if (has(i)) q = *reinterpret_cast<const uint4*>(row + at(i));
            w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
        }
    }
    __device__ __forceinline__ void init(const NormBwdParams& p, int t_, int threads_) {
        t = t_;
        threads = threads_;
        chunks = (int)(p.C / 8);
        load(p.w, ww);
#pragma unroll
        for (int i = 0; i < 8 * NV; ++i) dw[i] = 0.0f;
    }
    // This thread's part of sum g h rstd.
    __device__ __forceinline__ float dot(const uint32_t* dy, const uint32_t* h, float rstd) const {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) {
            s = __fmaf_rn(__fmul_rn(bf16lo(dy[i]), bf16lo(ww[i])), __fmul_rn(bf16lo(h[i]), rstd), s);
            s = __fmaf_rn(__fmul_rn(bf16hi(dy[i]), bf16hi(ww[i])), __fmul_rn(bf16hi(h[i]), rstd), s);
        }
        return s;
    }
    // dx of the row (c = the row's sum / C) and its share of dw.
    __device__ __forceinline__ void finish(const NormBwdParams& p, int64_t row, const uint32_t* dy, const uint32_t* h,
                                           const uint32_t* dh, float rstd, float c) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint32_t out[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = 4 * i + j;
                float d[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float dyv = b ? bf16hi(dy[k]) : bf16lo(dy[k]);
                    const float hr = __fmul_rn(b ? bf16hi(h[k]) : bf16lo(h[k]), rstd);
                    dw[2 * k + b] = __fmaf_rn(dyv, hr, dw[2 * k + b]);
                    const float v = __fmaf_rn(-hr, c, __fmul_rn(dyv, b ? bf16hi(ww[k]) : bf16lo(ww[k])));
                    d[b] = p.dh != nullptr ? __fmaf_rn(rstd, v, b ? bf16hi(dh[k]) : bf16lo(dh[k])) : __fmul_rn(rstd, v);
                }
                out[j] = norm_pack(d[0], d[1]);
            }
            if (has(i))
                *chk(reinterpret_cast<uint4*>(p.dx + row * p.lddx + at(i)), p.dx, rows_extent(p.R, p.C, p.lddx)) =
                    make_uint4(out[0], out[1], out[2], out[3]);
        }
    }
    __device__ __forceinline__ void write_dw(const NormBwdParams& p, int64_t owner, int64_t owners) const {
#pragma unroll
        for (int i = 0; i < 2 * NV; ++i)
            if (has(i / 2))
                *chk(reinterpret_cast<float4*>(p.dw_partials + owner * p.C + at(i / 2) + 4 * (i & 1)), p.dw_partials,
                     owners * p.C * 4) = make_float4(dw[4 * i], dw[4 * i + 1], dw[4 * i + 2], dw[4 * i + 3]);
    }
};

// C <= 512: a row belongs to one warp, loads straight to registers, the next
// row's before this row's sum is joined.
template <int NV>
__global__ void __launch_bounds__(128, 4) rmsnorm_bwd_warp_kernel(const NormBwdParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t owners = (int64_t)gridDim.x * 4, first = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    NormBwdThread<NV> th;
    th.init(p, lane, 32);
    uint32_t dy[4 * NV], h[4 * NV], dh[4 * NV], dy1[4 * NV], h1[4 * NV], dh1[4 * NV];
    float rstd = 0.0f, rstd1 = 0.0f;
    auto fetch = [&](int64_t row) {
        th.load(p.dy + row * p.lddy, dy1);
        th.load(p.h + row * p.ldh, h1);
        if (p.dh != nullptr) th.load(p.dh + row * p.lddh, dh1);
        rstd1 = p.rstd[row];
    };
    if (first < p.R) fetch(first);
    for (int64_t row = first; row < p.R; row += owners) {
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) {
            dy[i] = dy1[i];
            h[i] = h1[i];
            dh[i] = dh1[i];
        }
        rstd = rstd1;
        if (row + owners < p.R) fetch(row + owners);
        float s = th.dot(dy, h, rstd);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        th.finish(p, row, dy, h, dh, rstd, __fmul_rn(s, p.inv_c));
    }
    th.write_dw(p, first, owners);
}

// C > 512: a row belongs to one CTA of C / 16 threads. Rows arrive by bulk
// copies into a ring of p.stages shared-memory stages (dy, h and, if given, dh of
// one row each), so that several rows per SM are in flight without registers
// to hold them: measured on 16384 x 4096, 187 us with the rows loaded to
// registers when they are due, see the host code for the figure with the ring.
template <int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) rmsnorm_bwd_ring_kernel(const NormBwdParams p) {
    extern __shared__ __align__(1024) uint8_t dyn_smem[];
    __shared__ uint64_t full[kNormMaxStages];
    __shared__ float red[2][32];
    __shared__ int dead;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const uint32_t row_bytes = (uint32_t)p.C * 2, parts = p.dh != nullptr ? 3 : 2;
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 1);
        fence_mbarrier_init();
        dead = 0;
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    auto fetch = [&](int64_t row, int s) {  // one thread
        uint8_t* d = dyn_smem + s * parts * row_bytes;
        mbar_arrive_expect_tx(&full[s], parts * row_bytes);
        bulk_load(d, p.dy + row * p.lddy, row_bytes, &full[s]);
        bulk_load(d + row_bytes, p.h + row * p.ldh, row_bytes, &full[s]);
        if (p.dh != nullptr) bulk_load(d + 2 * row_bytes, p.dh + row * p.lddh, row_bytes, &full[s]);
    };
    if (threadIdx.x == 0)
        for (int s = 0; s < p.stages && blockIdx.x + (int64_t)s * gridDim.x < p.R; ++s)
            fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
    NormBwdThread<NV> th;
    th.init(p, threadIdx.x, blockDim.x);
    float rstd1 = blockIdx.x < p.R ? p.rstd[blockIdx.x] : 0.0f;
    int s = 0, parity = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < p.R; row += gridDim.x, parity ^= 1) {
        const float rstd = rstd1;
        if (row + gridDim.x < p.R) rstd1 = p.rstd[row + gridDim.x];
        if (!mbar_wait(&full[s], phase)) dead = 1;  // seen by all behind the barrier
        const uint16_t* d = reinterpret_cast<const uint16_t*>(dyn_smem + s * parts * row_bytes);
        uint32_t dy[4 * NV], h[4 * NV], dh[4 * NV];
        th.load(d, dy);
        th.load(d + p.C, h);
        if (p.dh != nullptr) th.load(d + 2 * p.C, dh);
        float sum = th.dot(dy, h, rstd);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) red[parity][warp] = sum;
        __syncthreads();  // the sums are written, and the stage is read
        if (dead) break;
        if (threadIdx.x == 0 && row + (int64_t)p.stages * gridDim.x < p.R) fetch(row + (int64_t)p.stages * gridDim.x, s);
        sum = red[parity][0];
        for (int w = 1; w < warps; ++w) sum += red[parity][w];
        th.finish(p, row, dy, h, dh, rstd, __fmul_rn(sum, p.inv_c));
        if (++s == p.stages) {
            s = 0;
            phase ^= 1u;
        }
    }
    th.write_dw(p, blockIdx.x, gridDim.x);
}

// dw[c] (+)= the sum of column c of the n partial rows, in a fixed order: 32
// columns per CTA, 32 threads per column.
__global__ void __launch_bounds__(1024) norm_dw_reduce_kernel(const float* partials, int n, int64_t C, float* dw,
                                                              int accumulate) {
    __shared__ float red[32][33];
    const int col = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + col;
    pdl_wait();
    pdl_launch_dependents();
    float s = 0.0f;
    if (c < C) {
#pragma unroll 8
        for (int r = part; r < n; r += 32) s += partials[(int64_t)r * C + c];
    }
    red[part][col] = s;
    __syncthreads();
    // warp w joins column w's 32 parts
    s = red[col][part];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int64_t cw = (int64_t)blockIdx.x * 32 + part;
    if (col == 0 && cw < C) *chk(dw + cw, dw, C * 4) = accumulate ? __fadd_rn(dw[cw], s) : s;
}

// Threads of a CTA and CTAs for R rows of C columns: as many as the SMs hold
// at once, at most `most` row owners (0: no such limit).
void norm_grid(int64_t R, int64_t C, int sms, int64_t most, int* threads, int* grid) {
    const bool warp_row = C <= kNormWarpRowC;
    const int64_t t = (C / kNormElems + (C % kNormElems != 0) + 31) / 32 * 32;
    const int64_t per_cta = warp_row ? 4 : 1;
    *threads = warp_row ? 128 : (int)t;
    int64_t g = (R + per_cta - 1) / per_cta;
    const int64_t fit = (int64_t)sms * std::max(1, 512 / *threads);
    g = std::min(g, fit);
    if (most > 0) g = std::min(g, most / per_cta);
    *grid = g < 1 ? 1 : (int)g;
}

template <int NH, bool QUANT>
cudaError_t launch_norm_fwd_t(const NormParams& p, int threads, int grid, cudaStream_t s) {
    const cudaError_t e =
        p.C <= kNormWarpRowC
            ? launch_pdl(rmsnorm_fwd_kernel<NH, QUANT, true>, dim3(grid), dim3(threads), 0, s, p)
            : launch_pdl(rmsnorm_fwd_kernel<NH, QUANT, false>, dim3(grid), dim3(threads), 0, s, p);
    count_launch();
    return e;
}

}  // namespace

cudaError_t launch_rmsnorm_fwd(NormParams p, int nh, bool quant, float* amax, int sms, int* n_partials,
                               cudaStream_t s) {
    int threads = 0, grid = 0;
    norm_grid(quant ? (p.R + 127) / 128 * 128 : p.R, p.C, sms, nh >= 0 && !quant ? kMaxAmaxPartials : 0, &threads, &grid);
    if (grid == 1) p.amax_out = amax;  // one CTA's maximum is the tensor's
    if (n_partials != nullptr) *n_partials = grid;
    if (quant) {
        switch (nh) {
            case 0: return launch_norm_fwd_t<0, true>(p, threads, grid, s);
            case 16: return launch_norm_fwd_t<16, true>(p, threads, grid, s);
            default: return launch_norm_fwd_t<32, true>(p, threads, grid, s);
        }
    }
    switch (nh) {
        case -1: return launch_norm_fwd_t<-1, false>(p, threads, grid, s);
        case 0: return launch_norm_fwd_t<0, false>(p, threads, grid, s);
        case 16: return launch_norm_fwd_t<16, false>(p, threads, grid, s);
        default: return launch_norm_fwd_t<32, false>(p, threads, grid, s);
    }
}

int64_t norm_bwd_partial_rows(int64_t R) { return std::min<int64_t>((R + 3) / 4 * 4, kMaxNormPartials); }

cudaError_t launch_rmsnorm_bwd(NormBwdParams p, float* dw, int accumulate, int sms, cudaStream_t s) {
    cudaError_t e;
    int owners;
    if (p.C <= 512) {
        const int grid = (int)std::min<int64_t>((p.R + 3) / 4, std::min(4 * sms, kMaxNormPartials / 4));
        owners = 4 * grid;
        auto run = [&](auto* kern) { return launch_pdl(kern, dim3(grid), dim3(128), 0, s, p); };
        e = p.C <= 256 ? run(rmsnorm_bwd_warp_kernel<1>)
                       : run(rmsnorm_bwd_warp_kernel<2>);
    } else {
        // 512 threads per SM, and its shared memory shared out among their rings
        const int threads = (int)((p.C + 511) / 512 * 32);
        const int per_sm = std::max(1, 512 / threads);
        const int stage = (p.dh != nullptr ? 3 : 2) * (int)p.C * 2;
        p.stages = std::min(kNormMaxStages, kNormRingBytes / per_sm / stage);
        owners = (int)std::min<int64_t>(p.R, std::min(per_sm * sms, kMaxNormPartials));
        auto run = [&](auto* kern) {
            const cudaError_t a = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormRingBytes);
            if (a != cudaSuccess) return a;
            return launch_pdl(kern, dim3(owners), dim3(threads), (size_t)(p.stages * stage), s, p);
        };
        e = threads <= 512 ? run(rmsnorm_bwd_ring_kernel<2, 512>) : run(rmsnorm_bwd_ring_kernel<2, 1024>);
    }
    count_launch();
    if (e != cudaSuccess) return e;
    e = launch_pdl(norm_dw_reduce_kernel, dim3((unsigned)((p.C + 31) / 32)), dim3(1024), 0, s,
                   static_cast<const float*>(p.dw_partials), owners, p.C, dw, accumulate);
    count_launch();
    return e;
}

}  // namespace qfp4
