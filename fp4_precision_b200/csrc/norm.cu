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
// registers between the sum and its use. A row belongs to one CTA, or, narrow
// ones, to one warp. Forward, a thread holds 16 or 32 elements of it, whole
// Hadamard groups and blocks, so that the rotation needs no shuffles; backward
// 16, and the weight gradient of its columns. CTAs are persistent: the weight
// is loaded once, and rows arrive ahead of their turn, forward in registers,
// backward (wide ones) by bulk copies into a ring in shared memory.
#include "qfp4_device.cuh"
#include "qfp4_internal.h"

namespace qfp4 {
namespace {

constexpr int kNormWarpRowC = 512;  // up to this many columns a row belongs to one warp (backward)
constexpr int kNormMaxStages = 4;   // rows in flight per CTA
constexpr int kNormRingBytes = 192 * 1024;

// 32 bytes of one thread, whole DRAM sectors in one instruction (32-byte aligned).
__device__ __forceinline__ void ldg256(const void* p, uint32_t* w) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void stg256(void* p, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
                 : "memory");
}

// A thread's part of a row: chunks t and (NCH = 2) t + threads of G elements.
template <int G, int NCH>
struct NormChunks {
    static constexpr int WORDS = G / 2 * NCH;
    int tpr, t;  // threads per row, this thread's index among them
    int chunks;  // chunks in a row
    bool wide;   // rows are 32-byte aligned
    __device__ __forceinline__ bool has(int i) const { return t + i * tpr < chunks; }
    __device__ __forceinline__ int at(int i) const { return (t + i * tpr) * G; }
    // packed bf16 pairs; chunks past the row are zero
    __device__ __forceinline__ void load(const uint16_t* row, uint32_t* w) const {
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int v = 0; v < G / 16; ++v) {
                uint32_t* d = w + i * (G / 2) + 8 * v;
                const uint16_t* src = row + at(i) + 16 * v;
                if (!has(i)) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) d[k] = 0;
                } else if (wide) {
                    ldg256(src, d);
                } else {
                    const uint4 q0 = reinterpret_cast<const uint4*>(src)[0], q1 = reinterpret_cast<const uint4*>(src)[1];
                    d[0] = q0.x; d[1] = q0.y; d[2] = q0.z; d[3] = q0.w;
                    d[4] = q1.x; d[5] = q1.y; d[6] = q1.z; d[7] = q1.w;
                }
            }
    }
    __device__ __forceinline__ void store(uint16_t* row, const uint32_t* w, const void* base, int64_t extent) const {
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int v = 0; v < G / 16; ++v) {
                const uint32_t* d = w + i * (G / 2) + 8 * v;
                uint16_t* dst = row + at(i) + 16 * v;
                if (!has(i)) continue;
                if (wide) {
                    stg256(chk(dst, base, extent, 32), d);
                } else {
                    uint4* q = reinterpret_cast<uint4*>(dst);
                    *chk(q, base, extent) = make_uint4(d[0], d[1], d[2], d[3]);
                    *chk(q + 1, base, extent) = make_uint4(d[4], d[5], d[6], d[7]);
                }
            }
    }
};

__device__ __forceinline__ uint32_t norm_pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ int64_t rows_extent(int64_t R, int64_t C, int64_t ld) { return R <= 0 ? 0 : ((R - 1) * ld + C) * 2; }

// ---- forward -------------------------------------------------------------------
// NH: -1 no amax, else the Hadamard size of the amax or (QUANT) of the MXFP4
// quantization.
template <int NH, bool QUANT>
constexpr int kNormChunk = (QUANT || NH == 32) ? 32 : 16;  // whole Hadamard groups and MXFP4 blocks
template <int NH, bool QUANT, int NCH>
struct NormFwd {
    static constexpr int G = kNormChunk<NH, QUANT>;
    static_assert(G == 16 || NCH == 1, "32 elements at most");
    using Chunks = NormChunks<G, NCH>;
    static constexpr int WORDS = Chunks::WORDS;
    Chunks ch;
    uint32_t ww[WORDS];
    float amax = 0.0f;

    // h = x + r of this thread's elements, stored, and the sum of its squares.
    __device__ __forceinline__ double residual(const NormParams& p, int64_t row, const uint32_t* xw, const uint32_t* rw,
                                               uint32_t* hw) const {
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            hw[i] = p.res != nullptr ? norm_pack(__fadd_rn(bf16lo(xw[i]), bf16lo(rw[i])),
                                                 __fadd_rn(bf16hi(xw[i]), bf16hi(rw[i])))
                                     : xw[i];
            const double a = bf16lo(hw[i]), b = bf16hi(hw[i]);
            ss = __fma_rn(a, a, ss);
            ss = __fma_rn(b, b, ss);
        }
        if (p.h != nullptr) ch.store(p.h + row * p.ldh, hw, p.h, rows_extent(p.R, p.C, p.ldh));
        return ss;
    }
    // y from h and the row's sum of squares, stored; in hw's place.
    __device__ __forceinline__ void normalize(const NormParams& p, int64_t row, uint32_t* hw, double ss) const {
        const float rstd = (float)rsqrt(ss * p.inv_c + p.eps);
        if (ch.t == 0) *chk(p.rstd + row, p.rstd, p.R * 4) = rstd;
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
            hw[i] = norm_pack(__fmul_rn(__fmul_rn(bf16lo(hw[i]), rstd), bf16lo(ww[i])),
                              __fmul_rn(__fmul_rn(bf16hi(hw[i]), rstd), bf16hi(ww[i])));
        if (!QUANT || p.y != nullptr) ch.store(p.y + row * p.ldy, hw, p.y, rows_extent(p.R, p.C, p.ldy));
    }
    // y's amax or quantization; rows from R on (up to the scale atom's 128) get
    // zero scales.
    __device__ __forceinline__ void output(const NormParams& p, int64_t row, const uint32_t* yw) {
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
                    uint32_t x = yw[i];
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
            for (int i = 0; i < NCH; ++i) {
                float v[G];
#pragma unroll
                for (int k = 0; k < G / 2; ++k) {
                    uint32_t x = yw[i * (G / 2) + k];
                    if (NH > 0 && p.signs != 0u) x ^= Grp::sign_mask(p.signs, k);
                    v[2 * k] = bf16lo(x);
                    v[2 * k + 1] = bf16hi(x);
                }
                if (ch.has(i)) amax = rot_abs_max<NH, G>(amax, v);
            }
        }
    }
    // The CTA's maximum; c * max |y| = max |c * y|.
    __device__ __forceinline__ void finish(const NormParams& p, float* red_max) {
        if constexpr (!QUANT && NH >= 0) {
            if constexpr (NH > 0) amax = __fmul_rn(amax, had_norm<NH>());
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            if ((threadIdx.x & 31) == 0) red_max[threadIdx.x >> 5] = amax;
            __syncthreads();
            if (threadIdx.x == 0) {
                for (int w = 1; w < (int)(blockDim.x >> 5); ++w) amax = fmaxf(amax, red_max[w]);
                *chk(p.amax_out + blockIdx.x, p.amax_out, (int64_t)gridDim.x * 4) = amax;
            }
        }
    }
    // Rows to walk: with the quantization up to the scale atom's 128.
    static __device__ __forceinline__ int64_t rows(const NormParams& p) {
        return QUANT ? (p.R + 127) / 128 * 128 : p.R;
    }
};

// A row belongs to one warp (WARP_ROW) or one CTA; its loads go straight to
// registers, the next row's before this row's sum is joined.
template <int NH, bool QUANT, int NCH, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? 128 : 512) rmsnorm_fwd_kernel(const NormParams p) {
    using Fwd = NormFwd<NH, QUANT, NCH>;
    __shared__ double red[2][16];
    __shared__ float red_max[16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t owners = WARP_ROW ? (int64_t)gridDim.x * warps : gridDim.x;
    const int64_t first = WARP_ROW ? (int64_t)blockIdx.x * warps + warp : blockIdx.x;
    Fwd f;
    f.ch = typename Fwd::Chunks{WARP_ROW ? 32 : (int)blockDim.x, WARP_ROW ? lane : (int)threadIdx.x,
                                (int)(p.C / Fwd::G), p.wide != 0};
    pdl_wait();  // the previous kernel's writes are visible (and its reads done)
    pdl_launch_dependents();
    uint32_t xw[Fwd::WORDS], rw[Fwd::WORDS];
    f.ch.load(p.w, f.ww);
    if (first < p.R) {
        f.ch.load(p.x + first * p.ldx, xw);
        if (p.res != nullptr) f.ch.load(p.res + first * p.ldres, rw);
    }
    if (QUANT && blockIdx.x == 0 && threadIdx.x == 0) *chk(p.q_tensor_scale, p.q_tensor_scale, 4) = 1.0f;
    int parity = 0;
    for (int64_t row = first; row < Fwd::rows(p); row += owners, parity ^= 1) {
        uint32_t hw[Fwd::WORDS];
        if (row < p.R) {
            double ss = f.residual(p, row, xw, rw, hw);
            if (row + owners < p.R) {
                f.ch.load(p.x + (row + owners) * p.ldx, xw);
                if (p.res != nullptr) f.ch.load(p.res + (row + owners) * p.ldres, rw);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if constexpr (!WARP_ROW) {
                // two halves in turn: the next row's sums do not overtake this one's
                if (lane == 0) red[parity][warp] = ss;
                __syncthreads();
                ss = red[parity][0];
                for (int w = 1; w < warps; ++w) ss += red[parity][w];
            }
            f.normalize(p, row, hw, ss);
        }
        f.output(p, row, hw);
    }
    f.finish(p, red_max);
}

// Rows in flight: a ring of p.stages shared-memory stages that bulk copies
// fill with one row each of up to three tensors.
struct NormRing {
    uint64_t full[kNormMaxStages];
    int dead[2];  // a wait ran out; for even and odd rows in turn, so that a
                  // thread a row ahead does not change what this row's threads read
    __device__ __forceinline__ void init(int stages) {
        if (threadIdx.x == 0) {
            for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
            fence_mbarrier_init();
            dead[0] = dead[1] = 0;
        }
        __syncthreads();
    }
};

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
// row's before this row's sum is joined. There are as many warps as rows of
// weight gradients (kMaxNormPartials, four per SM), so that one CTA runs on an SM
// and few rows are on their way: 65536 x 256 with dh, floor 21 us, takes 81.
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
// to hold them (16384 x 4096 with dh, 537 MB: 78 us and 4.5 for the weight
// gradient's join; 187 with the rows loaded to registers when they are due).
// Past 8192 columns a CTA has more than 512 threads, at most 64 registers each,
// and spills: 4096 x 16384 with dh, floor 82 us, takes 163.
template <int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) rmsnorm_bwd_ring_kernel(const NormBwdParams p) {
    extern __shared__ __align__(1024) uint8_t dyn_smem[];
    __shared__ NormRing ring;
    __shared__ float red[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const uint32_t row_bytes = (uint32_t)p.C * 2, parts = p.dh != nullptr ? 3 : 2;
    ring.init(p.stages);
    pdl_wait();
    pdl_launch_dependents();
    auto fetch = [&](int64_t row, int s) {  // one thread
        uint8_t* d = dyn_smem + s * parts * row_bytes;
        mbar_arrive_expect_tx(&ring.full[s], parts * row_bytes);
        bulk_load(d, p.dy + row * p.lddy, row_bytes, &ring.full[s]);
        bulk_load(d + row_bytes, p.h + row * p.ldh, row_bytes, &ring.full[s]);
        if (p.dh != nullptr) bulk_load(d + 2 * row_bytes, p.dh + row * p.lddh, row_bytes, &ring.full[s]);
    };
    if (threadIdx.x == 0)
        for (int s = 0; s < p.stages && blockIdx.x + (int64_t)s * gridDim.x < p.R; ++s)
            fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
    NormBwdThread<NV> th;
    th.init(p, threadIdx.x, blockDim.x);
    float rstd1 = blockIdx.x < p.R ? p.rstd[blockIdx.x] : 0.0f;
    int s = 0, parity = 0;
    uint32_t phase = 0;
    int64_t row = blockIdx.x;
    for (; row < p.R; row += gridDim.x, parity ^= 1) {
        const float rstd = rstd1;
        if (row + gridDim.x < p.R) rstd1 = p.rstd[row + gridDim.x];
        if (!mbar_wait(&ring.full[s], phase)) ring.dead[parity] = 1;  // seen by all behind the barrier
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
        if (ring.dead[parity]) break;
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
    if (row < p.R && threadIdx.x == 0) {
        // a wait ran out: no copy of the rows ahead lands after this CTA exits
        const int64_t done = (row - blockIdx.x) / gridDim.x, rows = (p.R - 1 - blockIdx.x) / gridDim.x + 1;
        drain_loads(ring.full, nullptr, p.stages, (int)min(done + p.stages, rows));
    }
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

// Stages of one CTA's ring, per_sm CTAs sharing the SM's shared memory.
int norm_stages(int per_sm, int stage_bytes) { return std::min(kNormMaxStages, kNormRingBytes / per_sm / stage_bytes); }

template <typename Kern, typename Params>
cudaError_t launch_norm_ring(Kern kern, int grid, int threads, int smem, const Params& p, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormRingBytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(grid), dim3(threads), (size_t)smem, s, p);
}

// Where a row is a CTA's, 768 threads per SM with 16 elements each (63 to 70
// registers) and 512 with 32 (115 to 128), and no more CTAs than amax partials.
// Measured with the amax on 16384 x 4096, 537 MB: 84 us with 16 elements and
// 32-byte accesses; 91 with 32 elements, 90 with 32 and 16-byte accesses; 99
// with the rows in a ring as in the backward pass (here half the traffic is
// stores, and more loads in flight delay them). Into MXFP4, 4099 x 5120, 179 MB:
// 31 us, 35 with 16-byte accesses.
// Where a row is a warp's the same counts are launched, but a thread takes 100
// registers with the 16-point amax and 138 to 147 with 32 elements: four of the
// six CTAs per SM run at once, or three of the four, and the rest after them.
// 65536 x 256, floors 21 and 22 us: 47 with the amax, 93 into MXFP4.
template <int NH, bool QUANT, int NCH>
cudaError_t launch_norm_fwd_t(NormParams p, float* amax, int sms, int* n_partials, cudaStream_t s) {
    constexpr int G = kNormChunk<NH, QUANT>;
    const int64_t rows = QUANT ? (p.R + 127) / 128 * 128 : p.R;
    const bool warp_row = p.C <= 32 * G;
    const int threads = warp_row ? 128 : (int)((p.C + G * NCH * 32 - 1) / (G * NCH * 32) * 32);
    const int per_sm = std::max(1, (G * NCH == 16 ? 768 : 512) / threads);
    int64_t grid = std::min<int64_t>(warp_row ? (rows + 3) / 4 : rows, (int64_t)per_sm * sms);
    if (NH >= 0 && !QUANT) grid = std::min<int64_t>(grid, kMaxAmaxPartials);
    if (grid == 1) p.amax_out = amax;  // one CTA's maximum is the tensor's
    if (n_partials != nullptr) *n_partials = (int)grid;
    const cudaError_t e =
        warp_row ? launch_pdl(rmsnorm_fwd_kernel<NH, QUANT, 1, true>, dim3((unsigned)grid), dim3(threads), 0, s, p)
                 : launch_pdl(rmsnorm_fwd_kernel<NH, QUANT, NCH, false>, dim3((unsigned)grid), dim3(threads), 0, s, p);
    count_launch();
    return e;
}

}  // namespace

cudaError_t launch_rmsnorm_fwd(const NormParams& p, int nh, bool quant, float* amax, int sms, int* n_partials,
                               cudaStream_t s) {
    if (quant) {
        switch (nh) {
            case 0: return launch_norm_fwd_t<0, true, 1>(p, amax, sms, n_partials, s);
            case 16: return launch_norm_fwd_t<16, true, 1>(p, amax, sms, n_partials, s);
            default: return launch_norm_fwd_t<32, true, 1>(p, amax, sms, n_partials, s);
        }
    }
    if (nh == 32) return launch_norm_fwd_t<32, false, 1>(p, amax, sms, n_partials, s);
    // at most 512 threads: two chunks of 16 each from 8192 columns on
    if (p.C <= 8192) {
        switch (nh) {
            case -1: return launch_norm_fwd_t<-1, false, 1>(p, amax, sms, n_partials, s);
            case 0: return launch_norm_fwd_t<0, false, 1>(p, amax, sms, n_partials, s);
            default: return launch_norm_fwd_t<16, false, 1>(p, amax, sms, n_partials, s);
        }
    }
    switch (nh) {
        case -1: return launch_norm_fwd_t<-1, false, 2>(p, amax, sms, n_partials, s);
        case 0: return launch_norm_fwd_t<0, false, 2>(p, amax, sms, n_partials, s);
        default: return launch_norm_fwd_t<16, false, 2>(p, amax, sms, n_partials, s);
    }
}

int64_t norm_bwd_partial_rows(int64_t R) { return std::min<int64_t>((R + 3) / 4 * 4, kMaxNormPartials); }

cudaError_t launch_rmsnorm_bwd(NormBwdParams p, float* dw, int accumulate, int sms, cudaStream_t s) {
    cudaError_t e;
    int owners;
    if (p.C <= kNormWarpRowC) {
        const int grid = (int)std::min<int64_t>((p.R + 3) / 4, std::min(4 * sms, kMaxNormPartials / 4));
        owners = 4 * grid;
        auto run = [&](auto* kern) { return launch_pdl(kern, dim3(grid), dim3(128), 0, s, p); };
        e = p.C <= 256 ? run(rmsnorm_bwd_warp_kernel<1>) : run(rmsnorm_bwd_warp_kernel<2>);
    } else {
        const int threads = (int)((p.C + 511) / 512 * 32), per_sm = std::max(1, 512 / threads);
        const int stage = (p.dh != nullptr ? 3 : 2) * (int)p.C * 2;
        p.stages = norm_stages(per_sm, stage);
        owners = (int)std::min<int64_t>(p.R, std::min(per_sm * sms, kMaxNormPartials));
        e = threads <= 512 ? launch_norm_ring(rmsnorm_bwd_ring_kernel<2, 512>, owners, threads, p.stages * stage, p, s)
                           : launch_norm_ring(rmsnorm_bwd_ring_kernel<2, 1024>, owners, threads, p.stages * stage, p, s);
    }
    count_launch();
    if (e != cudaSuccess) return e;
    e = launch_pdl(norm_dw_reduce_kernel, dim3((unsigned)((p.C + 31) / 32)), dim3(1024), 0, s,
                   static_cast<const float*>(p.dw_partials), owners, p.C, dw, accumulate);
    count_launch();
    return e;
}

}  // namespace qfp4
