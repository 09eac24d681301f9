// Root-mean-square norm with the residual's addition, and its gradients, for
// gfx950: the rows the routed block reads.
//
// Forward, per token row of d values:
//   s = x + r (r the residual; none: s = x),  rstd = (mean(s^2) + eps)^(-1/2),
//   y = s rstd w.
// s is the float32 sum; its squares are summed in float64; s and y are each
// rounded once, where they are stored, and y is computed from the float32 s.  For MXFP8 blocks the
// row's E4M3 codes and E8M0 scales are written in the same pass.  They are the
// codes of the stored bf16 y (the arithmetic of quantize_mxfp8_kernel), so an
// MXFP8 forward fed with them is bit for bit the forward fed with y; the extra
// rounding is half a bf16 step, 2^-8 of a value, against the 2^-4 of the E4M3
// rounding that follows.
//
// Backward, with n = s rstd and u = dy w:
//   ds = rstd (u - n mean(u n)) + dsum,   dw = sum over tokens of dy n.
//
// All of it is bound by HBM: every tensor is read or written once.  A row
// stays in registers between its reduction and its output.  Forward, T = 32768,
// d = 2048, MXFP8 rows with residual and codes: 94 us, 6.5 TB/s; backward,
// T = 16384, d = 4096, bf16 with dsum: 98 us, 5.5 TB/s (a 2 GiB copy runs at
// 4.9 TB/s on the same card).
#include <algorithm>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

template <bool BF>
__device__ __forceinline__ void unpack16(const u32x4& w, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            v[i] = __uint_as_float(w[i]);
        }
    }
}

template <bool BF>
__device__ __forceinline__ u32x4 pack16(const float (&v)[8]) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = BF ? pack_bf16x2(v[2 * i], v[2 * i + 1]) : __float_as_uint(v[i]);
    return w;
}

// Sum over the TPR threads of a row, the same on each (fixed order: butterfly
// in the wave, then the waves in order).
template <int TPR, typename V>
__device__ __forceinline__ V row_sum(V v, V* red) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < TPR / 64; ++w) v += red[w];
    }
    return v;
}

struct NormArgs {
    const u32x4* x;
    const u32x4* r;      // NULL: no residual
    const u32x4* w;
    u32x4* sum;          // optional
    u32x4* y;            // optional with q
    uint2* q;            // optional: E4M3 codes [T][d]
    uint32_t* qs;        // with q: scale dwords [T][d / 128]
    float* rstd;         // optional
    int T, chunks;       // 16-byte chunks of a row
    double inv_d;
    float eps;
};

// TPR threads per row (a wave, or a workgroup of 256); CH chunks per thread
// stay in registers, chunks past TPR CH of a longer row are read again.  A wave
// takes rows of up to two chunks a lane (T = 8000, d = 1024, bf16: 10.9 us, a
// workgroup a row 14.5); with four (T = 32768, d = 2048: 97 us against 93) or
// eight (T = 16384, d = 4096: 103 against 94) too few waves cover the loads.
template <bool BF, int TPR, int CH, bool NT>
__global__ __launch_bounds__(256) void norm_kernel(NormArgs a) {
    constexpr int NV = BF ? 8 : 4;
    __shared__ double red[4];
    const int lt = threadIdx.x % TPR;
    const int t = blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    if (t >= a.T) return;   // whole waves (TPR 64), or never (one row per workgroup)
    const size_t row = (size_t)t * a.chunks;
    float v[CH][8];
    u32x4 xr[CH], rr[CH];
#pragma unroll
    for (int g = 0; g < CH; ++g) {
        const int c = min(lt + TPR * g, a.chunks - 1);   // clamped chunks are loaded, not used
        xr[g] = stream_load<NT>(a.x + row + c);
        if (a.r) rr[g] = stream_load<NT>(a.r + row + c);
    }
    double ss = 0.0;
#pragma unroll
    for (int g = 0; g < CH; ++g) {
        unpack16<BF>(xr[g], v[g]);
        if (a.r) {
            float rv[8];
            unpack16<BF>(rr[g], rv);
#pragma unroll
            for (int i = 0; i < NV; ++i) v[g][i] += rv[i];
        }
        if (lt + TPR * g < a.chunks) {
#pragma unroll
            for (int i = 0; i < NV; ++i) ss = fma((double)v[g][i], (double)v[g][i], ss);
        }
    }
    auto load_sum = [&](int c, float (&o)[8]) {
        unpack16<BF>(a.x[row + c], o);
        if (a.r) {
            float rv[8];
            unpack16<BF>(a.r[row + c], rv);
#pragma unroll
            for (int i = 0; i < NV; ++i) o[i] += rv[i];
        }
    };
    for (int c = lt + TPR * CH; c < a.chunks; c += TPR) {
        float o[8];
        load_sum(c, o);
#pragma unroll
        for (int i = 0; i < NV; ++i) ss = fma((double)o[i], (double)o[i], ss);
    }
    // The row times a power of two, sc, that brings its mean square to [1, 4): the root, its reciprocal and s w stay in
    // float32's range for every row of finite values.  rstd of it as two floats (one step of Newton's method from the
    // rounded root), and y from them and the two halves of s w: y is the float32 nearest to the exact value for the
    // float32 s, so that a code or a scale at a rounding border is that value's too.  (What the addition of a residual
    // rounds away, up to 2^-24 of s, is left out: with it carried into y the rows of one chunk a thread took longer,
    // 32768 x 2048 with codes 99.7 us instead of 92.5, 8000 x 1024 13.3 instead of 10.5.)  Four more operations a value
    // than s rstd w, hidden behind the loads (32768 x 2048 with codes: 94 us, without the one for sc 93).
    const double ms = row_sum<TPR>(ss, red) * a.inv_d + a.eps;
    const int ex = (int)((unsigned long long)__double_as_longlong(ms) >> 52) - 1023;   // ms >= 0
    const int k = min(max(ex >> 1, -126), 126);
    const float sc = __uint_as_float((uint32_t)(127 - k) << 23);
    const double msc = ms * __longlong_as_double((long long)(1023 - 2 * k) << 52);
    const float mh = (float)msc, ml = (float)(msc - mh);
    const float r0 = 1.0f / sqrtf(mh), r2 = r0 * r0;
    const float re = fmaf(-mh, r2, 1.0f) - fmaf(mh, fmaf(r0, r0, -r2), ml * r2);
    const float corr = fabsf(re) < 1e-5f ? 0.5f * r0 * re : 0.f;   // 0: a mean square of 0, infinity or NaN
    const float rstd = r0 + corr, rl = corr != 0.f ? (r0 - rstd) + corr : 0.f;
    if (a.rstd && lt == 0) a.rstd[t] = rstd * sc;
    auto emit = [&](int c, const float (&s)[8]) {
        if (a.sum) stream_store<NT>(a.sum + row + c, pack16<BF>(s));
        float wv[8], o[8];
        unpack16<BF>(a.w[c], wv);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float n = s[i] * sc, p = n * wv[i];
            o[i] = fmaf(p, rstd, fmaf(p, rl, fmaf(n, wv[i], -p) * rstd));
        }
        const u32x4 yp = pack16<BF>(o);
        if (a.y) stream_store<NT>(a.y + row + c, yp);
        if constexpr (BF) {
            if (a.q) {   // d % 128 == 0: 16 lanes hold one 128-wide slice, 4 lanes one block of 32
                float f[8];
                unpack16<true>(yp, f);
                float amax = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
                amax = fmaxf(amax, __shfl_xor(amax, 1));
                amax = fmaxf(amax, __shfl_xor(amax, 2));
                const int se = mx_shared_exp(amax);
                const float inv = mx_inv_scale(se);
                a.q[row + c] = make_uint2(e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                                          e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
                uint32_t sw = (uint32_t)(se + 127) << (8 * ((c >> 2) & 3));
                sw |= __shfl_xor(sw, 4);
                sw |= __shfl_xor(sw, 8);
                if ((c & 15) == 0) a.qs[(size_t)t * (a.chunks / 16) + (c >> 4)] = sw;
            }
        }
    };
#pragma unroll
    for (int g = 0; g < CH; ++g)
        if (lt + TPR * g < a.chunks) emit(lt + TPR * g, v[g]);
    for (int c = lt + TPR * CH; c < a.chunks; c += TPR) {
        float o[8];
        load_sum(c, o);
        emit(c, o);
    }
}

// ----------------------------------------------------------------------------- backward

struct NormBwdArgs {
    const u32x4* dy;
    const u32x4* dsum;   // NULL: none
    const u32x4* s;
    const u32x4* w;
    const float* rstd;
    u32x4* ds;
    float* part;         // [blocks][d] partial weight gradients (row kernel)
    int T, chunks, rows; // rows per workgroup group of TPR threads
    float inv_d;
};

// Rows of at most TPR CH chunks: a group of TPR threads walks `rows`
// consecutive rows, keeping its columns' weights and weight-gradient sums in
// registers; the workgroup's groups are added in order into one partial row.
// A workgroup per row once a row has more than two chunks a lane (a wave per
// row of 4096 bf16 values needs 370 registers: one wave a SIMD, 120 us against
// 111 at T = 16384); streams that exceed the caches non-temporal (111 -> 101);
// the next row requested before a row is summed (101 -> 98 with half as many
// workgroups; T = 32768, d = 2048: 106 -> 99; two rows ahead 104).
template <bool BF, int TPR, int CH, bool NT>
__global__ __launch_bounds__(256) void norm_bwd_kernel(NormBwdArgs a) {
    constexpr int NV = BF ? 8 : 4;
    constexpr int NG = 256 / TPR;
    __shared__ float red[2][4];
    extern __shared__ float acc_s[];   // NG > 1: [NG - 1][chunks][NV]
    const int lt = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    float wv[CH][8], dw[CH][8];
#pragma unroll
    for (int g = 0; g < CH; ++g) {
        unpack16<BF>(a.w[min(lt + TPR * g, a.chunks - 1)], wv[g]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[g][i] = 0.f;
    }
    const int t0 = (blockIdx.x * NG + grp) * a.rows, t1 = min(a.T, t0 + a.rows);
    u32x4 sn[CH], yn[CH], en[CH];   // the next row, in flight while this one is summed and stored
    float rn = 0.f;
    auto load = [&](int t) {
        const size_t row = (size_t)t * a.chunks;
#pragma unroll
        for (int g = 0; g < CH; ++g) {
            const int c = min(lt + TPR * g, a.chunks - 1);
            sn[g] = stream_load<NT>(a.s + row + c);
            yn[g] = stream_load<NT>(a.dy + row + c);
            if (a.dsum) en[g] = stream_load<NT>(a.dsum + row + c);
        }
        rn = a.rstd[t];
    };
    if (t0 < t1) load(t0);
    for (int t = t0; t < t1; ++t) {
        const size_t row = (size_t)t * a.chunks;
        u32x4 sr[CH], yr[CH], er[CH];
        const float rstd = rn;
#pragma unroll
        for (int g = 0; g < CH; ++g) {
            sr[g] = sn[g];
            yr[g] = yn[g];
            er[g] = en[g];
        }
        if (t + 1 < t1) load(t + 1);
        float dot = 0.f;
#pragma unroll
        for (int g = 0; g < CH; ++g) {
            float sv[8], yv[8];
            unpack16<BF>(sr[g], sv);
            unpack16<BF>(yr[g], yv);
            if (lt + TPR * g < a.chunks) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const float n = sv[i] * rstd;
                    dot = fmaf(yv[i] * wv[g][i], n, dot);
                    dw[g][i] = fmaf(yv[i], n, dw[g][i]);
                }
            }
        }
        // the waves' sums alternate between two slots, so a row's are not
        // overwritten before every wave has read them
        const float m = row_sum<TPR>(dot, red[t & 1]) * a.inv_d;
#pragma unroll
        for (int g = 0; g < CH; ++g) {
            const int c = lt + TPR * g;
            if (c >= a.chunks) continue;
            float sv[8], yv[8], ev[8], o[8];
            unpack16<BF>(sr[g], sv);
            unpack16<BF>(yr[g], yv);
            if (a.dsum) unpack16<BF>(er[g], ev);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                o[i] = rstd * (yv[i] * wv[g][i] - sv[i] * rstd * m);
                if (a.dsum) o[i] += ev[i];
            }
            stream_store<NT>(a.ds + row + c, pack16<BF>(o));
        }
    }
    if constexpr (NG > 1) {
        if (grp > 0) {
#pragma unroll
            for (int g = 0; g < CH; ++g) {
                const int c = lt + TPR * g;
                if (c >= a.chunks) continue;
#pragma unroll
                for (int i = 0; i < NV; ++i) acc_s[((size_t)(grp - 1) * a.chunks + c) * NV + i] = dw[g][i];
            }
        }
        __syncthreads();
    }
    if (grp == 0) {
#pragma unroll
        for (int g = 0; g < CH; ++g) {
            const int c = lt + TPR * g;
            if (c >= a.chunks) continue;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float v = dw[g][i];
                if constexpr (NG > 1) {
#pragma unroll
                    for (int w = 0; w < NG - 1; ++w) v += acc_s[((size_t)w * a.chunks + c) * NV + i];
                }
                a.part[((size_t)blockIdx.x * a.chunks + c) * NV + i] = v;
            }
        }
    }
}

// Longer rows: one workgroup per row, read twice; the weight gradient is the
// column kernel's.
template <bool BF>
__global__ __launch_bounds__(256) void norm_bwd_long_kernel(NormBwdArgs a) {
    constexpr int NV = BF ? 8 : 4;
    __shared__ float red[4];
    const int t = blockIdx.x;
    const size_t row = (size_t)t * a.chunks;
    const float rstd = a.rstd[t];
    float dot = 0.f;
    for (int c = threadIdx.x; c < a.chunks; c += 256) {
        float sv[8], yv[8], wv[8];
        unpack16<BF>(a.s[row + c], sv);
        unpack16<BF>(a.dy[row + c], yv);
        unpack16<BF>(a.w[c], wv);
#pragma unroll
        for (int i = 0; i < NV; ++i) dot = fmaf(yv[i] * wv[i], sv[i] * rstd, dot);
    }
    const float m = row_sum<256>(dot, red) * a.inv_d;
    for (int c = threadIdx.x; c < a.chunks; c += 256) {
        float sv[8], yv[8], wv[8], ev[8], o[8];
        unpack16<BF>(a.s[row + c], sv);
        unpack16<BF>(a.dy[row + c], yv);
        unpack16<BF>(a.w[c], wv);
        if (a.dsum) unpack16<BF>(a.dsum[row + c], ev);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            o[i] = rstd * (yv[i] * wv[i] - sv[i] * rstd * m);
            if (a.dsum) o[i] += ev[i];
        }
        a.ds[row + c] = pack16<BF>(o);
    }
}

// part[blockIdx.y][c] = sum over the block's rows of dy s rstd, one chunk of
// columns per thread.
template <bool BF>
__global__ __launch_bounds__(256) void norm_dweight_long_kernel(NormBwdArgs a) {
    constexpr int NV = BF ? 8 : 4;
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.chunks) return;
    float dw[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int t0 = blockIdx.y * a.rows, t1 = min(a.T, t0 + a.rows);
    for (int t = t0; t < t1; ++t) {
        float sv[8], yv[8];
        unpack16<BF>(a.s[(size_t)t * a.chunks + c], sv);
        unpack16<BF>(a.dy[(size_t)t * a.chunks + c], yv);
        const float rstd = a.rstd[t];
#pragma unroll
        for (int i = 0; i < NV; ++i) dw[i] = fmaf(yv[i], sv[i] * rstd, dw[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) a.part[((size_t)blockIdx.y * a.chunks + c) * NV + i] = dw[i];
}

// dw[c] = sum of part[0, n)[c]: 64 columns per workgroup, its 16 waves take
// the partial rows in turn and are added in order.
__global__ __launch_bounds__(1024) void norm_dweight_reduce_kernel(const float* __restrict__ part, int n, int d,
                                                                   float* __restrict__ dw) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    constexpr int kB = 32;   // all of a wave's rows at once (n <= 512)
    float s = 0.f;
    for (int b = wave; b < n; b += 16 * kB) {
        float v[kB];
#pragma unroll
        for (int u = 0; u < kB; ++u) v[u] = b + 16 * u < n ? part[(size_t)(b + 16 * u) * d + c] : 0.f;
#pragma unroll
        for (int u = 0; u < kB; ++u) s += v[u];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int w = 1; w < 16; ++w) s += red[w][lane];
        dw[c] = s;
    }
}

// How a backward of T rows of `chunks` 16-byte chunks runs.
struct NormBwdPlan {
    int tpr;      // threads per row: 64, 256, or 0 for the kernels of long rows
    int ch;       // chunks per thread
    int rows;     // rows per group
    int blocks;   // partial rows of the weight gradient
};

// Two workgroups per compute unit; one where a row takes a workgroup's threads
// more than once and the tensors pass the caches (T = 16384, d = 4096, bf16: 98 us
// against 102; T = 32768, d = 2048: 119 against 99).
constexpr int kNormPartials = 512;

NormBwdPlan norm_bwd_plan(int T, int chunks) {
    NormBwdPlan p{};
    if (chunks <= 64 * 2) {
        p.tpr = 64;
        p.ch = chunks <= 64 ? 1 : 2;
    } else if (chunks <= 256 * 4) {
        p.tpr = 256;
        p.ch = chunks <= 256 ? 1 : (chunks <= 512 ? 2 : 4);
    }
    const bool one = p.tpr == 256 && p.ch > 1 && past_caches((size_t)T * chunks * 16);
    const int groups = (one ? kNormPartials / 2 : kNormPartials) * (p.tpr == 64 ? 4 : 1);
    p.rows = (T + groups - 1) / groups;
    const int per_block = p.rows * (p.tpr == 64 ? 4 : 1);
    p.blocks = (T + per_block - 1) / per_block;
    return p;
}

template <bool BF, bool NT>
void launch_norm_t(const NormArgs& a, hipStream_t s) {
    const dim3 b(256), rows(a.T), waves((a.T + 3) / 4);
    if (a.chunks <= 64) hipLaunchKernelGGL((norm_kernel<BF, 64, 1, NT>), waves, b, 0, s, a);
    else if (a.chunks <= 128) hipLaunchKernelGGL((norm_kernel<BF, 64, 2, NT>), waves, b, 0, s, a);
    else if (a.chunks <= 256) hipLaunchKernelGGL((norm_kernel<BF, 256, 1, NT>), rows, b, 0, s, a);
    else if (a.chunks <= 512) hipLaunchKernelGGL((norm_kernel<BF, 256, 2, NT>), rows, b, 0, s, a);
    else hipLaunchKernelGGL((norm_kernel<BF, 256, 4, NT>), rows, b, 0, s, a);
}

template <bool BF, bool NT>
void launch_norm_bwd_rows(const NormBwdArgs& a, const NormBwdPlan& p, hipStream_t s) {
    const dim3 b(256), g(p.blocks);
    const size_t lds = p.tpr == 64 ? (size_t)3 * a.chunks * 16 * (BF ? 2 : 1) : 0;
    if (p.tpr == 64) {
        if (p.ch == 1) hipLaunchKernelGGL((norm_bwd_kernel<BF, 64, 1, NT>), g, b, lds, s, a);
        else hipLaunchKernelGGL((norm_bwd_kernel<BF, 64, 2, NT>), g, b, lds, s, a);
    } else {
        if (p.ch == 1) hipLaunchKernelGGL((norm_bwd_kernel<BF, 256, 1, NT>), g, b, 0, s, a);
        else if (p.ch == 2) hipLaunchKernelGGL((norm_bwd_kernel<BF, 256, 2, NT>), g, b, 0, s, a);
        else hipLaunchKernelGGL((norm_bwd_kernel<BF, 256, 4, NT>), g, b, 0, s, a);
    }
}

template <bool BF>
void launch_norm_bwd_t(const NormBwdArgs& a, const NormBwdPlan& p, hipStream_t s) {
    if (p.tpr == 0) {
        // the weight gradient first: ds may be dy
        hipLaunchKernelGGL((norm_dweight_long_kernel<BF>), dim3((a.chunks + 255) / 256, p.blocks), dim3(256), 0, s, a);
        hipLaunchKernelGGL((norm_bwd_long_kernel<BF>), dim3(a.T), dim3(256), 0, s, a);
    } else if (past_caches((size_t)a.T * a.chunks * 16)) {   // (T = 8000, d = 512, 8 MB: 11.3 us through them, 12.4 past them)
        launch_norm_bwd_rows<BF, true>(a, p, s);
    } else {
        launch_norm_bwd_rows<BF, false>(a, p, s);
    }
}

}  // namespace

hipError_t launch_norm(int act, const void* x, const void* residual, const void* weight, float eps, void* sum, void* y,
                       void* q, uint8_t* q_scale, float* rstd, int T, int d, hipStream_t s) {
    const bool bf = act != kF32;
    const NormArgs a{static_cast<const u32x4*>(x), static_cast<const u32x4*>(residual),
                     static_cast<const u32x4*>(weight), static_cast<u32x4*>(sum), static_cast<u32x4*>(y),
                     static_cast<uint2*>(q), reinterpret_cast<uint32_t*>(q_scale), rstd, T, d / (bf ? 8 : 4),
                     1.0 / d, eps};
    const bool nt = past_caches((size_t)T * a.chunks * 16);
    if (bf && nt) launch_norm_t<true, true>(a, s);
    else if (bf) launch_norm_t<true, false>(a, s);
    else if (nt) launch_norm_t<false, true>(a, s);
    else launch_norm_t<false, false>(a, s);
    return hipGetLastError();
}

size_t norm_bwd_part_bytes(int act, int T, int d) {
    return (size_t)norm_bwd_plan(T, d / (act == kF32 ? 4 : 8)).blocks * d * 4;
}

hipError_t launch_norm_bwd(int act, const void* dy, const void* dsum, const void* s_in, const void* weight,
                           const float* rstd, void* ds, float* dweight, float* part, int T, int d, hipStream_t s) {
    const bool bf = act != kF32;
    const int chunks = d / (bf ? 8 : 4);
    const NormBwdPlan p = norm_bwd_plan(T, chunks);
    const NormBwdArgs a{static_cast<const u32x4*>(dy), static_cast<const u32x4*>(dsum),
                        static_cast<const u32x4*>(s_in), static_cast<const u32x4*>(weight), rstd,
                        static_cast<u32x4*>(ds), part, T, chunks, p.rows, 1.0f / (float)d};
    if (bf) launch_norm_bwd_t<true>(a, p, s);
    else launch_norm_bwd_t<false>(a, p, s);
    hipLaunchKernelGGL(norm_dweight_reduce_kernel, dim3(d / 64), dim3(1024), 0, s, part, p.blocks, d, dweight);
    return hipGetLastError();
}

}  // namespace moe
