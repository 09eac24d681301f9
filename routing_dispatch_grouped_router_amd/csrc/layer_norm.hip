// Layer norm with the residual's addition, and its gradients, for gfx950: the
// rows the routed block reads in models that subtract a row's mean.
//
// Forward, per token row of d values:
//   s = x + r (r the residual; none: s = x),  mu = mean(s),
//   rstd = (mean((s - mu)^2) + eps)^(-1/2),   y = (s - mu) rstd w + b.
// s is the float32 sum.  The mean is summed first and the squares of s - mu
// after it, from the row in registers: a difference of two large sums would
// lose what a row with a mean far from zero has left.  Both sums and y are taken
// in float64 (behind the loads), so y is the float32 nearest to the exact value
// for that s before it is stored, and an E8M0 scale or a code at a border is that
// value's.  MXFP8 codes and scales are those of the stored bf16 y, as moe_norm
// writes them.
//
// Backward, with n = (s - mu) rstd and u = dy w:
//   ds = rstd (u - mean(u) - n mean(u n)) + dsum,
//   dw = sum over tokens of dy n,  db = sum over tokens of dy.
//
// All of it is bound by HBM: every tensor is read or written once.  Forward,
// T = 32768, d = 2048, MXFP8 rows with residual and codes: 100 us, 6.1 TB/s;
// T = 16384, d = 4096, bf16 with residual: 88 us; its backward with dsum 98 us,
// 5.5 TB/s (a 2 GiB copy runs at 4.9 TB/s on the same card).
// Slower forwards: mean and squares in one pass about a value of the row, with s
// exact in float64 and rows walked with the next in flight (fewer waves for more
// float64 conversions: 107-122 us); y in float32 and values near a bf16 border
// again in float64 (124 us).
#include <algorithm>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

template <int CTRL>
__device__ __forceinline__ double dpp_add(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint64_t o = (uint64_t)dpp_u32<CTRL>((uint32_t)(u >> 32)) << 32 | dpp_u32<CTRL>((uint32_t)u);
    return v + __longlong_as_double((long long)o);
}

// row_sum in float64, inside rows of 16 lanes by DPP operand modifiers (32768 x 2048 with codes: 101 -> 99.6 us).
template <int TPR>
__device__ __forceinline__ double row_sum64(double v, double* red) {
    v = dpp_add<0x140>(dpp_add<0x141>(dpp_add<0x4E>(dpp_add<0xB1>(v))));
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < TPR / 64; ++w) v += red[w];
    }
    return v;
}

struct LayerNormArgs {
    const u32x4* x;
    const u32x4* r;      // NULL: no residual
    const u32x4* w;
    const u32x4* b;      // NULL: no bias
    u32x4* sum;          // optional
    u32x4* y;            // optional with q
    uint2* q;            // optional: E4M3 codes [T][d]
    uint32_t* qs;        // with q: scale dwords [T][d / 128]
    float* mean;         // optional
    float* rstd;         // optional
    int T, chunks;       // 16-byte chunks of a row
    double d, inv_d, eps;
};

// TPR threads per row (a wave, or a workgroup of 256); CH chunks per thread
// stay in registers, chunks past TPR CH of a longer row are read again.
template <bool BF, int TPR, int CH, bool NT>
__global__ __launch_bounds__(256) void layer_norm_kernel(LayerNormArgs a) {
    constexpr int NV = BF ? 8 : 4;
    __shared__ double red[2][4];
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
    auto load_sum = [&](int c, float (&o)[8]) {
        unpack16<BF>(a.x[row + c], o);
        if (a.r) {
            float rv[8];
            unpack16<BF>(a.r[row + c], rv);
#pragma unroll
            for (int i = 0; i < NV; ++i) o[i] += rv[i];
        }
    };
    double total = 0.0;
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
            for (int i = 0; i < NV; ++i) total += (double)v[g][i];
        }
    }
    for (int c = lt + TPR * CH; c < a.chunks; c += TPR) {
        float o[8];
        load_sum(c, o);
#pragma unroll
        for (int i = 0; i < NV; ++i) total += (double)o[i];
    }
    const double mu = row_sum64<TPR>(total, red[0]) / a.d;   // a product with a rounded 1 / d misses a value that all share
    double squares = 0.0;
    auto add_squares = [&](const float (&s)[8]) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const double e = (double)s[i] - mu;
            squares = fma(e, e, squares);
        }
    };
#pragma unroll
    for (int g = 0; g < CH; ++g)
        if (lt + TPR * g < a.chunks) add_squares(v[g]);
    for (int c = lt + TPR * CH; c < a.chunks; c += TPR) {
        float o[8];
        load_sum(c, o);
        add_squares(o);
    }
    const double rstd = rsqrt(row_sum64<TPR>(squares, red[1]) * a.inv_d + a.eps);
    if (lt == 0) {
        if (a.mean) a.mean[t] = (float)mu;
        if (a.rstd) a.rstd[t] = (float)rstd;
    }
    auto emit = [&](int c, const float (&s)[8]) {
        if (a.sum) stream_store<NT>(a.sum + row + c, pack16<BF>(s));
        float wv[8], bv[8], o[8];
        unpack16<BF>(a.w[c], wv);
        if (a.b) unpack16<BF>(a.b[c], bv);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            o[i] = (float)fma(((double)s[i] - mu) * rstd, (double)wv[i], a.b ? (double)bv[i] : 0.0);
            // kept from being folded with the rounding to bf16: one conversion from float64 takes a dozen operations
            // (105 us instead of 101)
            asm volatile("" : "+v"(o[i]));
        }
        const u32x4 yp = pack16<BF>(o);
        if (a.y) stream_store<NT>(a.y + row + c, yp);
        if constexpr (BF) {
            if (a.q) store_mxfp8_chunk(yp, c, a.q + row, a.qs + (size_t)t * (a.chunks / 16));
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

struct LayerNormBwdArgs {
    const u32x4* dy;
    const u32x4* dsum;   // NULL: none
    const u32x4* s;
    const u32x4* w;
    const float* mean;
    const float* rstd;
    u32x4* ds;
    float* part;         // [blocks][2][d] partial gradients of weight and bias
    int T, chunks, rows; // rows per group of TPR threads
    float inv_d;
};

// The sums of a row over its TPR threads, both at once.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* red) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
        a += __shfl_xor(a, m);
        b += __shfl_xor(b, m);
    }
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = make_float2(a, b);
        __syncthreads();
        const float2 first = red[0];
        a = first.x;
        b = first.y;
#pragma unroll
        for (int w = 1; w < TPR / 64; ++w) {
            const float2 o = red[w];
            a += o.x;
            b += o.y;
        }
    }
    return make_float2(a, b);
}

// Rows of at most TPR CH chunks: a group of TPR threads walks `rows`
// consecutive rows, keeping its columns' weights and the gradients' sums in
// registers, the next row requested before a row is summed; the workgroup's
// groups are added in order into one partial row.
template <bool BF, int TPR, int CH, bool NT>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void layer_norm_bwd_kernel(LayerNormBwdArgs a) {
    constexpr int NV = BF ? 8 : 4;
    constexpr int NG = TPR > 256 ? 1 : 256 / TPR;
    __shared__ float2 red[2][TPR > 256 ? TPR / 64 : 4];
    extern __shared__ float acc_s[];   // NG > 1: [NG - 1][2][chunks][NV]
    const int lt = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    // eight waves a row, bf16: weights and rows stay packed until they are used, or the sums go to memory (43 registers;
    // 4096 x 16384 with dsum 175 us instead of 107)
    constexpr bool kPacked = BF && TPR == 512;
    u32x4 wr[CH];
    float wf[CH][8], dw[CH][8], db[CH][8];
#pragma unroll
    for (int g = 0; g < CH; ++g) {
        wr[g] = a.w[min(lt + TPR * g, a.chunks - 1)];
        if (!kPacked) unpack16<BF>(wr[g], wf[g]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[g][i] = db[g][i] = 0.f;
    }
    const int t0 = (blockIdx.x * NG + grp) * a.rows, t1 = min(a.T, t0 + a.rows);
    u32x4 sn[CH], yn[CH], en[CH];   // the next row, in flight while this one is summed and stored
    float mn = 0.f, rn = 0.f;
    auto load = [&](int t) {
        const size_t row = (size_t)t * a.chunks;
#pragma unroll
        for (int g = 0; g < CH; ++g) {
            const int c = min(lt + TPR * g, a.chunks - 1);
            sn[g] = stream_load<NT>(a.s + row + c);
            yn[g] = stream_load<NT>(a.dy + row + c);
            if (a.dsum) en[g] = stream_load<NT>(a.dsum + row + c);
        }
        mn = a.mean[t];
        rn = a.rstd[t];
    };
    if (t0 < t1) load(t0);
    for (int t = t0; t < t1; ++t) {
        const size_t row = (size_t)t * a.chunks;
        u32x4 sr[CH], yr[CH], er[CH];
        const float mean = mn, rstd = rn;
#pragma unroll
        for (int g = 0; g < CH; ++g) {
            sr[g] = sn[g];
            yr[g] = yn[g];
            er[g] = en[g];
        }
        if (t + 1 < t1) load(t + 1);
        float su = 0.f, sun = 0.f;
#pragma unroll
        for (int g = 0; g < CH; ++g) {
            float sv[8], yv[8], wp[8];
            unpack16<BF>(sr[g], sv);
            unpack16<BF>(yr[g], yv);
            if (kPacked) {
                asm volatile("" : "+v"(wr[g]));   // unpacked here, not once in front of the loop
                unpack16<BF>(wr[g], wp);
            }
            const float(&wv)[8] = kPacked ? wp : wf[g];
            if (lt + TPR * g < a.chunks) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const float n = (sv[i] - mean) * rstd, u = yv[i] * wv[i];
                    su += u;
                    sun = fmaf(u, n, sun);
                    dw[g][i] = fmaf(yv[i], n, dw[g][i]);
                    db[g][i] += yv[i];
                }
            }
        }
        // the waves' sums alternate between two slots, so a row's are not
        // overwritten before every wave has read them
        const float2 m = row_sum2<TPR>(su, sun, red[t & 1]);
        const float mu = m.x * a.inv_d, mun = m.y * a.inv_d;
#pragma unroll
        for (int g = 0; g < CH; ++g) {
            const int c = lt + TPR * g;
            if (c >= a.chunks) continue;
            float sv[8], yv[8], ev[8], o[8], wp[8];
            if (kPacked) asm volatile("" : "+v"(sr[g]), "+v"(yr[g]));
            unpack16<BF>(sr[g], sv);
            unpack16<BF>(yr[g], yv);
            if (kPacked) {
                asm volatile("" : "+v"(wr[g]));   // and these
                unpack16<BF>(wr[g], wp);
            }
            const float(&wv)[8] = kPacked ? wp : wf[g];
            if (a.dsum) unpack16<BF>(er[g], ev);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float n = (sv[i] - mean) * rstd;
                o[i] = rstd * (fmaf(yv[i], wv[i], -mu) - n * mun);
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
                for (int i = 0; i < NV; ++i) {
                    acc_s[((size_t)(2 * (grp - 1)) * a.chunks + c) * NV + i] = dw[g][i];
                    acc_s[((size_t)(2 * (grp - 1) + 1) * a.chunks + c) * NV + i] = db[g][i];
                }
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
                float v = dw[g][i], u = db[g][i];
                if constexpr (NG > 1) {
#pragma unroll
                    for (int w = 0; w < NG - 1; ++w) {
                        v += acc_s[((size_t)(2 * w) * a.chunks + c) * NV + i];
                        u += acc_s[((size_t)(2 * w + 1) * a.chunks + c) * NV + i];
                    }
                }
                a.part[((size_t)(2 * blockIdx.x) * a.chunks + c) * NV + i] = v;
                a.part[((size_t)(2 * blockIdx.x + 1) * a.chunks + c) * NV + i] = u;
            }
        }
    }
}

// Longer rows: one workgroup per row, read twice; the gradients of weight and
// bias are the column kernel's.
template <bool BF>
__global__ __launch_bounds__(256) void layer_norm_bwd_long_kernel(LayerNormBwdArgs a) {
    constexpr int NV = BF ? 8 : 4;
    __shared__ float2 red[4];
    const int t = blockIdx.x;
    const size_t row = (size_t)t * a.chunks;
    const float mean = a.mean[t], rstd = a.rstd[t];
    float su = 0.f, sun = 0.f;
    for (int c = threadIdx.x; c < a.chunks; c += 256) {
        float sv[8], yv[8], wv[8];
        unpack16<BF>(a.s[row + c], sv);
        unpack16<BF>(a.dy[row + c], yv);
        unpack16<BF>(a.w[c], wv);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float u = yv[i] * wv[i];
            su += u;
            sun = fmaf(u, (sv[i] - mean) * rstd, sun);
        }
    }
    const float2 m = row_sum2<256>(su, sun, red);
    const float mu = m.x * a.inv_d, mun = m.y * a.inv_d;
    for (int c = threadIdx.x; c < a.chunks; c += 256) {
        float sv[8], yv[8], wv[8], ev[8], o[8];
        unpack16<BF>(a.s[row + c], sv);
        unpack16<BF>(a.dy[row + c], yv);
        unpack16<BF>(a.w[c], wv);
        if (a.dsum) unpack16<BF>(a.dsum[row + c], ev);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float n = (sv[i] - mean) * rstd;
            o[i] = rstd * (fmaf(yv[i], wv[i], -mu) - n * mun);
            if (a.dsum) o[i] += ev[i];
        }
        a.ds[row + c] = pack16<BF>(o);
    }
}

// part[blockIdx.y][0 and 1][c] = sums over the block's rows of dy n and dy, one
// chunk of columns per thread.
template <bool BF>
__global__ __launch_bounds__(256) void layer_norm_columns_kernel(LayerNormBwdArgs a) {
    constexpr int NV = BF ? 8 : 4;
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.chunks) return;
    float dw[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, db[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int t0 = blockIdx.y * a.rows, t1 = min(a.T, t0 + a.rows);
    for (int t = t0; t < t1; ++t) {
        float sv[8], yv[8];
        unpack16<BF>(a.s[(size_t)t * a.chunks + c], sv);
        unpack16<BF>(a.dy[(size_t)t * a.chunks + c], yv);
        const float mean = a.mean[t], rstd = a.rstd[t];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            dw[i] = fmaf(yv[i], (sv[i] - mean) * rstd, dw[i]);
            db[i] += yv[i];
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        a.part[((size_t)(2 * blockIdx.y) * a.chunks + c) * NV + i] = dw[i];
        a.part[((size_t)(2 * blockIdx.y + 1) * a.chunks + c) * NV + i] = db[i];
    }
}

// dw[c] and db[c] from the n partial rows of 2 d columns: 64 columns per
// workgroup, its 16 waves take the partial rows in turn and are added in order.
__global__ __launch_bounds__(1024) void layer_norm_reduce_kernel(const float* __restrict__ part, int n, int d,
                                                                 float* __restrict__ dw, float* __restrict__ db) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    constexpr int kB = 32;   // all of a wave's rows at once (n <= 512)
    float s = 0.f;
    for (int b = wave; b < n; b += 16 * kB) {
        float v[kB];
#pragma unroll
        for (int u = 0; u < kB; ++u) v[u] = b + 16 * u < n ? part[(size_t)(b + 16 * u) * 2 * d + c] : 0.f;
#pragma unroll
        for (int u = 0; u < kB; ++u) s += v[u];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int w = 1; w < 16; ++w) s += red[w][lane];
        if (c < d) dw[c] = s;      // d % 64 == 0: a workgroup's columns are all of one gradient
        else if (db) db[c - d] = s;
    }
}

// Small batches: every gradient in one launch.  Workgroups [0, row_blocks) take
// a row per wave; the others 8 chunks of columns each over all rows, 128 rows at
// a time (8 lanes a row, so that they read whole 128-byte pieces), eight loads
// of a lane in flight, and add the row lanes in a fixed order.  s and dy are
// read twice, from the caches.  `first`: the workgroup that blockIdx.x 0 is.
template <bool BF>
__global__ __launch_bounds__(1024) void layer_norm_bwd_small_kernel(LayerNormBwdArgs a, int row_blocks, int first,
                                                                    float* __restrict__ dw, float* __restrict__ db) {
    constexpr int NV = BF ? 8 : 4;
    constexpr int CH = 2;
    __shared__ float red[2][16][8 * NV];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = blockIdx.x + first;
    if (b < row_blocks) {
        const int t = b * 16 + wave;
        if (t >= a.T) return;
        const size_t row = (size_t)t * a.chunks;
        const float mean = a.mean[t], rstd = a.rstd[t];
        float sv[CH][8], yv[CH][8], wv[CH][8], ev[CH][8];
#pragma unroll
        for (int g = 0; g < CH; ++g) {
            const int c = min(lane + 64 * g, a.chunks - 1);
            unpack16<BF>(a.s[row + c], sv[g]);
            unpack16<BF>(a.dy[row + c], yv[g]);
            unpack16<BF>(a.w[c], wv[g]);
            if (a.dsum) unpack16<BF>(a.dsum[row + c], ev[g]);
        }
        float su = 0.f, sun = 0.f;
#pragma unroll
        for (int g = 0; g < CH; ++g) {
            if (lane + 64 * g >= a.chunks) continue;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float u = yv[g][i] * wv[g][i];
                su += u;
                sun = fmaf(u, (sv[g][i] - mean) * rstd, sun);
            }
        }
        const float2 m = row_sum2<64>(su, sun, nullptr);
        const float mu = m.x * a.inv_d, mun = m.y * a.inv_d;
#pragma unroll
        for (int g = 0; g < CH; ++g) {
            if (lane + 64 * g >= a.chunks) continue;
            float o[8];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float n = (sv[g][i] - mean) * rstd;
                o[i] = rstd * (fmaf(yv[g][i], wv[g][i], -mu) - n * mun);
                if (a.dsum) o[i] += ev[g][i];
            }
            a.ds[row + lane + 64 * g] = pack16<BF>(o);
        }
        return;
    }
    const int c = 8 * (b - row_blocks) + (lane & 7);   // chunks % 8 == 0
    float w[NV], u[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) w[i] = u[i] = 0.f;
    constexpr int kB = 8;
    for (int r = threadIdx.x >> 3; r < a.T; r += 128 * kB) {
        u32x4 sr[kB], yr[kB];
        float mean[kB], rstd[kB];
#pragma unroll
        for (int j = 0; j < kB; ++j) {
            const int t = min(r + 128 * j, a.T - 1);
            sr[j] = a.s[(size_t)t * a.chunks + c];
            yr[j] = a.dy[(size_t)t * a.chunks + c];
            mean[j] = a.mean[t];
            rstd[j] = a.rstd[t];
        }
#pragma unroll
        for (int j = 0; j < kB; ++j) {
            if (r + 128 * j >= a.T) continue;
            float sv[8], yv[8];
            unpack16<BF>(sr[j], sv);
            unpack16<BF>(yr[j], yv);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                w[i] = fmaf(yv[i], (sv[i] - mean[j]) * rstd[j], w[i]);
                u[i] += yv[i];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int m = 8; m <= 32; m <<= 1) {
            w[i] += __shfl_xor(w[i], m);
            u[i] += __shfl_xor(u[i], m);
        }
        if (lane < 8) {
            red[0][wave][NV * lane + i] = w[i];
            red[1][wave][NV * lane + i] = u[i];
        }
    }
    __syncthreads();
    const int k = threadIdx.x / (8 * NV), col = threadIdx.x % (8 * NV);
    if (k < 2) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += red[k][i][col];
        float* out = k ? db : dw;
        if (out) out[8 * NV * (b - row_blocks) + col] = v;
    }
}

// How a backward of T rows of `chunks` 16-byte chunks runs.
struct LayerNormBwdPlan {
    bool small;   // one launch; the rest describes the other kernels
    int tpr;      // threads per row: 64, 256, 512, or 0 for the kernels of long rows
    int ch;       // chunks per thread
    int rows;     // rows per group
    int blocks;   // partial rows
};

// Two workgroups per compute unit; one where a row takes a workgroup's threads
// more than once (T = 16384, d = 4096, bf16 with dsum: 98 us against 106;
// T = 2048: 18.3 against 19.9; T = 32768, d = 2048, once: 118 against 100).
constexpr int kPartials = 512;

// Rows of up to two chunks a lane that take one launch (a second costs 3 us:
// T = 777, d = 192, float32: 7.1 us against 9.6 through the binding, T = 1000,
// d = 1024, bf16: 7.6 against 9.8; T = 2000, d = 1024: 13.1 against 12.2).
constexpr int kSmallRows = 1024;

LayerNormBwdPlan layer_norm_bwd_plan(int T, int chunks) {
    LayerNormBwdPlan p{};
    p.small = chunks <= 128 && T <= kSmallRows;
    if (chunks <= 64 * 2) {
        p.tpr = 64;
        p.ch = chunks <= 64 ? 1 : 2;
    } else if (chunks <= 256 * 4) {
        p.tpr = 256;
        p.ch = chunks <= 256 ? 1 : (chunks <= 512 ? 2 : 4);
    } else if (chunks <= 512 * 4) {   // (T = 4096, d = 8192, float32 with dsum: 101 us, by the kernels of long rows 184)
        p.tpr = 512;
        p.ch = 4;
    }
    const int groups = p.tpr == 64 ? kPartials * 4 : (p.ch > 1 ? kPartials / 2 : kPartials);
    p.rows = (T + groups - 1) / groups;
    const int per_block = p.rows * (p.tpr == 64 ? 4 : 1);
    p.blocks = (T + per_block - 1) / per_block;
    return p;
}

template <bool BF, bool NT>
void launch_forward(const LayerNormArgs& a, hipStream_t s) {
    const dim3 b(256), rows(a.T), waves((a.T + 3) / 4);
    if (a.chunks <= 64) hipLaunchKernelGGL((layer_norm_kernel<BF, 64, 1, NT>), waves, b, 0, s, a);
    else if (a.chunks <= 128) hipLaunchKernelGGL((layer_norm_kernel<BF, 64, 2, NT>), waves, b, 0, s, a);
    else if (a.chunks <= 256) hipLaunchKernelGGL((layer_norm_kernel<BF, 256, 1, NT>), rows, b, 0, s, a);
    else if (a.chunks <= 512) hipLaunchKernelGGL((layer_norm_kernel<BF, 256, 2, NT>), rows, b, 0, s, a);
    else hipLaunchKernelGGL((layer_norm_kernel<BF, 256, 4, NT>), rows, b, 0, s, a);
}

template <bool BF, bool NT>
void launch_bwd_rows(const LayerNormBwdArgs& a, const LayerNormBwdPlan& p, hipStream_t s) {
    const dim3 b(256), g(p.blocks);
    const size_t lds = p.tpr == 64 ? (size_t)6 * a.chunks * 16 * (BF ? 2 : 1) : 0;
    if (p.tpr == 64) {
        if (p.ch == 1) hipLaunchKernelGGL((layer_norm_bwd_kernel<BF, 64, 1, NT>), g, b, lds, s, a);
        else hipLaunchKernelGGL((layer_norm_bwd_kernel<BF, 64, 2, NT>), g, b, lds, s, a);
    } else if (p.tpr == 512) {
        hipLaunchKernelGGL((layer_norm_bwd_kernel<BF, 512, 4, NT>), g, dim3(512), 0, s, a);
    } else {
        if (p.ch == 1) hipLaunchKernelGGL((layer_norm_bwd_kernel<BF, 256, 1, NT>), g, b, 0, s, a);
        else if (p.ch == 2) hipLaunchKernelGGL((layer_norm_bwd_kernel<BF, 256, 2, NT>), g, b, 0, s, a);
        else hipLaunchKernelGGL((layer_norm_bwd_kernel<BF, 256, 4, NT>), g, b, 0, s, a);
    }
}

template <bool BF>
void launch_bwd(const LayerNormBwdArgs& a, const LayerNormBwdPlan& p, hipStream_t s) {
    if (p.tpr == 0) {
        // the columns' sums first: ds may be dy
        hipLaunchKernelGGL((layer_norm_columns_kernel<BF>), dim3((a.chunks + 255) / 256, p.blocks), dim3(256), 0, s, a);
        hipLaunchKernelGGL((layer_norm_bwd_long_kernel<BF>), dim3(a.T), dim3(256), 0, s, a);
    } else if (past_caches((size_t)a.T * a.chunks * 16)) {
        launch_bwd_rows<BF, true>(a, p, s);
    } else {
        launch_bwd_rows<BF, false>(a, p, s);
    }
}

}  // namespace

hipError_t launch_layer_norm(int act, const void* x, const void* residual, const void* weight, const void* bias,
                             float eps, void* sum, void* y, void* q, uint8_t* q_scale, float* mean, float* rstd, int T,
                             int d, hipStream_t s) {
    const bool bf = act != kF32;
    const LayerNormArgs a{static_cast<const u32x4*>(x), static_cast<const u32x4*>(residual),
                          static_cast<const u32x4*>(weight), static_cast<const u32x4*>(bias),
                          static_cast<u32x4*>(sum), static_cast<u32x4*>(y), static_cast<uint2*>(q),
                          reinterpret_cast<uint32_t*>(q_scale), mean, rstd, T, d / (bf ? 8 : 4), (double)d, 1.0 / d, eps};
    const bool nt = past_caches((size_t)T * a.chunks * 16);
    if (bf && nt) launch_forward<true, true>(a, s);
    else if (bf) launch_forward<true, false>(a, s);
    else if (nt) launch_forward<false, true>(a, s);
    else launch_forward<false, false>(a, s);
    return hipGetLastError();
}

size_t layer_norm_bwd_part_bytes(int act, int T, int d) {
    return (size_t)layer_norm_bwd_plan(T, d / (act == kF32 ? 4 : 8)).blocks * 2 * d * 4;
}

hipError_t launch_layer_norm_bwd(int act, const void* dy, const void* dsum, const void* s_in, const void* weight,
                                 const float* mean, const float* rstd, void* ds, float* dweight, float* dbias,
                                 float* part, int T, int d, hipStream_t s) {
    const bool bf = act != kF32;
    const int chunks = d / (bf ? 8 : 4);
    const LayerNormBwdPlan p = layer_norm_bwd_plan(T, chunks);
    const LayerNormBwdArgs a{static_cast<const u32x4*>(dy), static_cast<const u32x4*>(dsum),
                             static_cast<const u32x4*>(s_in), static_cast<const u32x4*>(weight), mean, rstd,
                             static_cast<u32x4*>(ds), part, T, chunks, p.rows, 1.0f / (float)d};
    if (p.small) {
        const int rows = (T + 15) / 16, cols = chunks / 8;
        auto go = [&](int first, int n) {
            if (bf) hipLaunchKernelGGL((layer_norm_bwd_small_kernel<true>), dim3(n), dim3(1024), 0, s, a, rows, first, dweight, dbias);
            else hipLaunchKernelGGL((layer_norm_bwd_small_kernel<false>), dim3(n), dim3(1024), 0, s, a, rows, first, dweight, dbias);
        };
        if (ds != dy) {
            go(0, rows + cols);
        } else {   // the columns' sums before dy is written over
            go(rows, cols);
            go(0, rows);
        }
        return hipGetLastError();
    }
    if (bf) launch_bwd<true>(a, p, s);
    else launch_bwd<false>(a, p, s);
    hipLaunchKernelGGL(layer_norm_reduce_kernel, dim3((dbias ? 2 : 1) * d / 64), dim3(1024), 0, s, part, p.blocks, d,
                       dweight, dbias);
    return hipGetLastError();
}

}  // namespace moe
