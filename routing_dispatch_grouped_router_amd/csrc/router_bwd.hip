// Gradients of the router's product logits = x W_r from dense logit gradients
// dL [T][E] (float32), for gfx950:
//   dx[t] = add[t] + sum_e dL[t][e] W_r[:, e],   dW_r = x^T dL.
// The block's own router gradient is zero outside the selected experts and is
// summed sparsely (backward.hip); the gradient of a loss on the router's
// probabilities touches every expert, so here both are dense products.
//
// Both run on the bf16 matrix cores.  A float32 operand is written as three
// bfloat16 terms whose sum has its 24 bits (v = v1 + v2 + v3, each the rounded
// remainder of the ones before), and the products of terms i, j with
// i + j <= 4 are summed in the float32 accumulators: what is left out is below
// 2^-24 of the product.  dL is always split, x and W_r only for float32 blocks.
// The terms of an infinity, and of a value that rounds past bfloat16's largest,
// are not its sum but NaN, and a zero remainder times an infinity is NaN too, so
// a sum that comes out NaN is taken again in float32 from the operands: it is
// then what the products give, +-inf or NaN.
#include <algorithm>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

// Three bfloat16 terms of eight float32 values, two at a time.
__device__ __forceinline__ void split3(const float (&v)[8], bf16x8 (&o)[3]) {
    u32x4 w[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const uint32_t u = pack_bf16x2(a, b);
            w[p][i] = u;
            a -= __uint_as_float(u << 16);
            b -= __uint_as_float(u & 0xFFFF0000u);
        }
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) o[p] = __builtin_bit_cast(bf16x8, w[p]);
}

// c += a b for operands of TA and TB terms (1 or 3), the smallest products first.
template <int TA, int TB>
__device__ __forceinline__ f32x4 mfma_terms(const bf16x8 (&a)[TA], const bf16x8 (&b)[TB], f32x4 c) {
#pragma unroll
    for (int n = 2; n >= 0; --n)
#pragma unroll
        for (int i = 0; i <= n; ++i)
            if (i < TA && n - i < TB) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[n - i], c, 0, 0, 0);
    return c;
}

// Eight consecutive values p[i .. i + 8) of a row whose last n are valid
// (zero past them), as operand terms.  vec: all eight valid or none, aligned.
template <bool BF>
__device__ __forceinline__ void load_terms(const void* p, size_t i, int n, bool vec, bf16x8 (&o)[BF ? 1 : 3]) {
    if constexpr (BF) {
        if (vec) {
            o[0] = n > 0 ? *reinterpret_cast<const bf16x8*>(static_cast<const uint16_t*>(p) + i)
                         : __builtin_bit_cast(bf16x8, (u32x4){0u, 0u, 0u, 0u});
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            o[0][j] = __builtin_bit_cast(__bf16, j < n ? static_cast<const uint16_t*>(p)[i + j] : (uint16_t)0);
    } else {
        float v[8];
        const float* f = static_cast<const float*>(p);
        if (vec) {
            f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
            if (n > 0) {
                lo = *reinterpret_cast<const f32x4*>(f + i);
                hi = *reinterpret_cast<const f32x4*>(f + i + 4);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = lo[j];
                v[4 + j] = hi[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = j < n ? f[i + j] : 0.f;
        }
        split3(v, o);
    }
}

// The same with all eight valid and 16 bytes aligned.
template <bool BF>
__device__ __forceinline__ void load_terms_full(const void* p, uint32_t i, bf16x8 (&o)[BF ? 1 : 3]) {
    if constexpr (BF) {
        o[0] = *reinterpret_cast<const bf16x8*>(static_cast<const uint16_t*>(p) + i);
    } else {
        const f32x4 lo = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
        const f32x4 hi = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i + 4);
        const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        split3(v, o);
    }
}

// Value i of an operand in memory.
template <bool BF>
__device__ __forceinline__ float value_at(const void* p, size_t i) {
    return BF ? bf16_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

// Whether one of N sums is NaN.
template <int N>
__device__ __forceinline__ bool any_nan(const float (&v)[N]) {
    bool n = false;
#pragma unroll
    for (int i = 0; i < N; ++i) n |= v[i] != v[i];
    return n;
}

// Whether a lane of the wave has a NaN sum.
template <int M, int N>
__device__ __forceinline__ bool wave_nan(const f32x4 (&acc)[M][N]) {
    bool n = false;
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) n |= any_nan({acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]});
    return __any(n);
}

// v[j] = sum_e dL[t][e] W_r[c + j][e] in float32, for the rows whose sums of terms are NaN.
template <bool BF>
__device__ __forceinline__ void row_product(const float* dL, const void* w, int t, int c, int E, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll 1
    for (int e = 0; e < E; ++e) {
        const float g = dL[(size_t)t * E + e];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = fmaf(g, value_at<BF>(w, (size_t)(c + j) * E + e), v[j]);
    }
}

}  // namespace

// dx: a workgroup owns 64 tokens and 256 columns, a wave 32 by 128 of them, as
// 16 x 16 blocks: M = tokens, N = columns, K = experts.  Column n of the wave's
// block j is column 8 n + j, so that a lane's eight blocks hold 8 consecutive
// columns of a token and sixteen lanes 128: add is read and dx written in whole
// lines (a lane layout with a row per lane cost the memory pipe an access per
// lane: 1.7 times as long at T = 16384, d = 4096, E = 64, where this takes 64 us).
// Both operands pass through LDS in fragment order, 32 experts at a time, loaded
// in whole 64- and 128-byte pieces and split once for the workgroup; two buffers,
// the next experts' loads in flight during a step's products.  `add`: row t of add (pos NULL; requested
// before the products), or the sum of its rows pos[t][0 .. k), or nothing (NULL).
template <bool BF>
__global__ __launch_bounds__(256) void router_dx_kernel(const float* __restrict__ dL, const void* __restrict__ w,
                                                        const void* add, const int32_t* __restrict__ pos, int k,
                                                        void* dx, int T, int d, int E) {
    constexpr int TA = BF ? 1 : 3;
    constexpr int NC = BF ? 1 : 2;           // 16-byte chunks of 8 columns
    __shared__ u32x4 s_a[2][4][3][64];       // dL: [token block][term], lane (token m, experts 8 q ..) at 16 q + (m ^ 4 q)
    __shared__ u32x4 s_w[2][16][TA][64];     // W_r: [block][term], lane (column n, experts 8 q ..) at 16 q + (n ^ 4 q ^ j % 4)
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, q = lane >> 4;
    const int ncb = (d + 255) / 256, tb = blockIdx.x / ncb;
    const int t0 = tb * 64, c0 = (int)(blockIdx.x - tb * ncb) * 256;
    const int wt = t0 + 32 * (wave & 1), wc = c0 + 128 * (wave >> 1);
    const bool vec = (E & 7) == 0;
    const size_t row_chunks = (size_t)d / (BF ? 8 : 4), cb = (size_t)(wc + 8 * m) / (BF ? 8 : 4);
    const bool in_cols = wc + 8 * m < d;
    const u32x4* src = static_cast<const u32x4*>(add);

    // thread: experts 8 (tid % 4) .. of token tid / 4 and of columns tid / 4 + 64 i
    const int lr = tid >> 2, lq = tid & 3;
    // (uniform bases and 32-bit lane offsets, and a path without the test for the last expert: address and select
    // instructions held this kernel up: 8 % longer with a 64-bit offset and a test a load)
    const float* dl0 = dL + (size_t)t0 * E;
    const char* w0 = static_cast<const char*>(w) + (size_t)c0 * E * (BF ? 2 : 4);
    const uint32_t dlo = (uint32_t)min(lr, T - 1 - t0) * (uint32_t)E + 8 * lq;
    uint32_t wo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) wo[i] = (uint32_t)min(lr + 64 * i, d - 1 - c0) * (uint32_t)E + 8 * lq;
    bf16x8 ra[3], rw[4][TA];
    auto load = [&](int e0) {
        const int n = E - e0 - 8 * lq;
        const float* dle = dl0 + e0;
        const char* we = w0 + (size_t)e0 * (BF ? 2 : 4);
        if (vec && e0 + 32 <= E) {   // no expert is past the last
            load_terms_full<false>(dle, dlo, ra);
#pragma unroll
            for (int i = 0; i < 4; ++i) load_terms_full<BF>(we, wo[i], rw[i]);
        } else {
            load_terms<false>(dle, dlo, n, vec, ra);
#pragma unroll
            for (int i = 0; i < 4; ++i) load_terms<BF>(we, wo[i], n, vec, rw[i]);
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int p = 0; p < 3; ++p)
            s_a[buf][lr >> 4][p][16 * lq + ((lr & 15) ^ (4 * lq))] = __builtin_bit_cast(u32x4, ra[p]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = lr + 64 * i, j = c & 7, n = (c >> 3) & 15;
#pragma unroll
            for (int p = 0; p < TA; ++p)
                s_w[buf][8 * (c >> 7) + j][p][16 * lq + (n ^ (4 * lq) ^ (j & 3))] = __builtin_bit_cast(u32x4, rw[i][p]);
        }
    };
    load(0);
    u32x4 base[2][4][NC];
    if (src && !pos) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = min(wt + 16 * mt + 4 * q + i, T - 1);
#pragma unroll
                for (int g = 0; g < NC; ++g) base[mt][i][g] = in_cols ? src[t * row_chunks + cb + g] : (u32x4){0u, 0u, 0u, 0u};
            }
    }
    f32x4 acc[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    int buf = 0;
    for (int e0 = 0; e0 < E; e0 += 32, buf ^= 1) {
        stage(buf);
        __syncthreads();   // also: every wave has left the buffer that is written next
        if (e0 + 32 < E) load(e0 + 32);
        bf16x8 a[2][3];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int p = 0; p < 3; ++p)
                a[mt][p] = __builtin_bit_cast(bf16x8, s_a[buf][2 * (wave & 1) + mt][p][16 * q + (m ^ (4 * q))]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            bf16x8 b[TA];
#pragma unroll
            for (int p = 0; p < TA; ++p)
                b[p] = __builtin_bit_cast(bf16x8, s_w[buf][8 * (wave >> 1) + j][p][16 * q + (m ^ (4 * q) ^ (j & 3))]);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) acc[mt][j] = mfma_terms<3, TA>(a[mt], b, acc[mt][j]);
        }
    }
    if (!in_cols) return;
    u32x4* dst = static_cast<u32x4*>(dx);
    auto value = [](const u32x4 (&c)[NC], int j) {   // value j of 8 in memory order
        return BF ? __uint_as_float((j & 1) ? (c[0][j / 2] & 0xFFFF0000u) : (c[0][j / 2] << 16))
                  : __uint_as_float(c[NC == 1 ? 0 : j / 4][j % 4]);
    };
    // row t: `b` or the gathered rows, plus the product's sums
    auto finish = [&](int t, const u32x4 (&b)[NC], const float (&sum)[8]) {
        float v[8];
        if (pos) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.f;
            for (int s = 0; s < k; ++s) {
                const size_t r = (size_t)pos[(size_t)t * k + s];
                u32x4 c[NC];
#pragma unroll
                for (int g = 0; g < NC; ++g) c[g] = src[r * row_chunks + cb + g];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += value(c, j);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = src ? value(b, j) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += sum[j];
#pragma unroll
        for (int g = 0; g < NC; ++g) {
            u32x4 o;
#pragma unroll
            for (int h = 0; h < 4; ++h)
                o[h] = BF ? pack_bf16x2(v[2 * h], v[2 * h + 1]) : __float_as_uint(v[4 * g + h]);
            dst[t * row_chunks + cb + g] = o;
        }
    };
    auto row_sums = [&](int mt, int i, float (&sum)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = acc[mt][j][i];
    };
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = wt + 16 * mt + 4 * q + i;
            float sum[8];
            row_sums(mt, i, sum);
            if (t < T) finish(t, base[mt][i], sum);
        }
    if (wave_nan(acc)) {   // those rows again (what was added is in base: dx may be add)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = wt + 16 * mt + 4 * q + i;
                float sum[8];
                row_sums(mt, i, sum);
                if (t >= T || !any_nan(sum)) continue;
                row_product<BF>(dL, w, t, wc + 8 * m, E, sum);
                finish(t, base[mt][i], sum);
            }
    }
}

// The same for bfloat16 blocks of at most 32 NS experts (two 32's fit the LDS
// of two workgroups) and rows added one for one: a workgroup keeps its 256
// columns of W_r in LDS and walks `rows` tokens, 64 at a time, the next tokens'
// dL and rows of add in flight during a tile's products.  55 us at T = 16384,
// d = 4096, E = 64, 4.9 TB/s (the kernel above: 64; through the caches 58, and
// dW_r, which reads x from them, 43 instead of 34); 17 us at T = 8192, d = 2048,
// E = 8 (19).
template <int NS, bool NT>
__global__ __launch_bounds__(256, 2) void router_dx_resident_kernel(const float* __restrict__ dL,
                                                                    const uint16_t* __restrict__ w, const u32x4* add,
                                                                    u32x4* dx, int T, int d, int E, int rows) {
    __shared__ u32x4 s_w[NS][16][64];
    __shared__ u32x4 s_a[2][NS][4][3][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, q = lane >> 4;
    const int ncb = (d + 255) / 256, tb = blockIdx.x / ncb, c0 = (int)(blockIdx.x - tb * ncb) * 256;
    const int ta = tb * rows, te = min(T, ta + rows);
    const int wc = c0 + 128 * (wave >> 1), lr = tid >> 2, lq = tid & 3;
    const bool vec = (E & 7) == 0, in_cols = wc + 8 * m < d;
    const uint32_t row_chunks = (uint32_t)d / 8, cb = (uint32_t)(wc + 8 * m) / 8;
    f32x4 la[NS][2];
    auto load_dl = [&](int t0) {
        const float* base = dL + (size_t)t0 * E;
        const uint32_t o = (uint32_t)min(lr, te - 1 - t0) * (uint32_t)E + 8 * lq;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const int n = E - 32 * s - 8 * lq;
            if (vec) {
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    la[s][g] = n > 0 ? *reinterpret_cast<const f32x4*>(base + (o + 32 * s + 4 * g)) : (f32x4){0.f, 0.f, 0.f, 0.f};
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) la[s][j / 4][j % 4] = j < n ? base[o + 32 * s + j] : 0.f;
            }
        }
    };
    u32x4 base[2][4];
    auto load_base = [&](int t0) {
        const u32x4* at = add + (size_t)t0 * row_chunks;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = min(32 * (wave & 1) + 16 * mt + 4 * q + i, te - 1 - t0);
                base[mt][i] = stream_load<NT>(at + ((uint32_t)t * row_chunks + (in_cols ? cb : 0u)));
            }
    };
    load_dl(ta);
    {
        const uint16_t* w0 = w + (size_t)c0 * E;
        bf16x8 rw[NS][4][1];
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                load_terms<true>(w0 + 32 * s, (size_t)min(lr + 64 * i, d - 1 - c0) * E + 8 * lq, E - 32 * s - 8 * lq, vec,
                                 rw[s][i]);
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = lr + 64 * i, j = c & 7, n = (c >> 3) & 15;
                s_w[s][8 * (c >> 7) + j][16 * lq + (n ^ (4 * lq) ^ (j & 3))] = __builtin_bit_cast(u32x4, rw[s][i][0]);
            }
    }
    if (add) load_base(ta);
    int buf = 0;
    for (int t0 = ta; t0 < te; t0 += 64, buf ^= 1) {
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const float v[8] = {la[s][0][0], la[s][0][1], la[s][0][2], la[s][0][3],
                                la[s][1][0], la[s][1][1], la[s][1][2], la[s][1][3]};
            bf16x8 o[3];
            split3(v, o);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                s_a[buf][s][lr >> 4][p][16 * lq + ((lr & 15) ^ (4 * lq))] = __builtin_bit_cast(u32x4, o[p]);
        }
        __syncthreads();   // also: every wave has left the buffer that is written next
        if (t0 + 64 < te) load_dl(t0 + 64);
        f32x4 acc[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            bf16x8 a[2][3];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    a[mt][p] = __builtin_bit_cast(bf16x8, s_a[buf][s][2 * (wave & 1) + mt][p][16 * q + (m ^ (4 * q))]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bf16x8 b[1] = {
                    __builtin_bit_cast(bf16x8, s_w[s][8 * (wave >> 1) + j][16 * q + (m ^ (4 * q) ^ (j & 3))])};
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) acc[mt][j] = mfma_terms<3, 1>(a[mt], b, acc[mt][j]);
            }
        }
        u32x4* dt = dx + (size_t)t0 * row_chunks;
        auto finish = [&](int t, const u32x4& b, const float (&sum)[8]) {   // row t0 + t: the row added, plus the sums
            u32x4 o;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const uint32_t c = add ? b[h] : 0u;
                o[h] = pack_bf16x2(__uint_as_float(c << 16) + sum[2 * h],
                                   __uint_as_float(c & 0xFFFF0000u) + sum[2 * h + 1]);
            }
            stream_store<NT>(dt + ((uint32_t)t * row_chunks + cb), o);
        };
        auto row_sums = [&](int mt, int i, float (&sum)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] = acc[mt][j][i];
        };
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 32 * (wave & 1) + 16 * mt + 4 * q + i;
                float sum[8];
                row_sums(mt, i, sum);
                if (in_cols && t0 + t < te) finish(t, base[mt][i], sum);
            }
        if (wave_nan(acc)) {   // those rows again (what was added is in base: dx may be add)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 32 * (wave & 1) + 16 * mt + 4 * q + i;
                    float sum[8];
                    row_sums(mt, i, sum);
                    if (!in_cols || t0 + t >= te || !any_nan(sum)) continue;
                    row_product<true>(dL, w, t0 + t, wc + 8 * m, E, sum);
                    finish(t, base[mt][i], sum);
                }
        }
        if (add && t0 + 64 < te) load_base(t0 + 64);
    }
}

// dW_r partials: a workgroup sums CT columns x 16 NT experts over a range of
// tokens, 32 at a time.  M = columns, N = experts, K = tokens.  The x tile is
// staged in LDS as blocks of 16 columns [32 tokens][16] (32-byte rows, blocks
// 32 bytes apart in the banks) and read transposed (ds_read_b64_tr_b16: 16
// lanes addressing rows r0 + L / 4 and columns 4 (L % 4) .. + 3 receive rows
// r0 .. r0 + 3 of column L); the dL operands are split once, by wave nt for
// experts 16 nt .. + 16, and shared through LDS.  LDS reads and the tiles'
// latency bound it, and a dL block is three times an x block, so with 64
// experts two waves share the columns and a wave's tile is 128 columns by 32
// experts (32 us at T = 16384, d = 4096, E = 64, and 7 for the ranges' sum; the
// two 14 % longer with 32 by 64).  Two buffers, and the loads of the next PD
// tiles in flight (7 % longer with loads behind a test for the range's end,
// where a tile waits for every later one's; as much with two workgroups joined
// in one, for half as many partial sums).
template <bool BF, int NT, int CT>
__global__ __launch_bounds__(256, 2) void router_dw_kernel(const float* __restrict__ dL, const void* __restrict__ x,
                                                        float* __restrict__ part, int T, int d, int E, int rows) {
    typedef short v4s __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4s* lp;
    constexpr int TA = BF ? 1 : 3;
    constexpr int kTile = 32 * 32 + 32;                 // bytes of a 16-column block, padded
    constexpr int NX = BF ? 1 : 2;                      // 16-byte loads of 8 columns
    constexpr int PD = BF && NT < 4 ? 4 : 2;            // (four tiles of 64 experts: 9 % longer)
    constexpr int XI = CT / 64;                         // 8-column items of a thread: 32 tokens x CT / 8 chunks
    constexpr int WE = NT == 4 ? 2 : 1, WC = 4 / WE;    // waves over the experts, over the columns
    constexpr int MT = CT / WC / 16, NW = NT / WE;      // a wave's blocks
    __shared__ __align__(16) char s_x[2][TA][CT / 16 * kTile];
    __shared__ u32x4 s_b[2][NT][3][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, q = lane >> 4;
    const int c0 = blockIdx.x * CT, e0 = blockIdx.y * 16 * NT;
    const int t0 = blockIdx.z * rows, t1 = min(T, t0 + rows);
    const int wm = MT * (wave % WC), wn = NW * (wave / WC);   // the wave's first blocks
    const size_t rowc = (size_t)d / (BF ? 8 : 4);       // 16-byte chunks of a row
    const int lt = tid / (CT / 8), lc = tid % (CT / 8); // loader: token lt + 2048 / CT i, columns 8 lc .. + 8
    f32x4 acc[MT][NW];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NW; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};

    u32x4 xr[PD][XI][NX];
    float br[PD][8];
    // this thread's columns and expert, clamped (what is past d or E is not stored)
    const uint32_t xc = (uint32_t)min(c0 + 8 * lc, d - 8) / (BF ? 8 : 4);
    const int be = min(e0 + 16 * min(wave, NT - 1) + m, E - 1);
    // A tile is the 32 rows from tb, or the range's last 32 if they end before tb + 32 (all of them if it is shorter):
    // every load is unconditional, so that a tile waits for its own loads alone, and stage() clears the other rows.
    const int nrow = min(32, t1 - t0), last = t1 - nrow;
    uint32_t xo[XI], bo[8];
#pragma unroll
    for (int i = 0; i < XI; ++i) xo[i] = (uint32_t)(min(lt + 2048 / CT * i, nrow - 1) * rowc) + xc;
#pragma unroll
    for (int j = 0; j < 8; ++j) bo[j] = (uint32_t)min(8 * q + j, nrow - 1) * (uint32_t)E + be;
    auto load = [&](int tb, u32x4 (&xr)[XI][NX], float (&br)[8]) {
        tb = min(tb, last);
        const u32x4* xt = static_cast<const u32x4*>(x) + (size_t)tb * rowc;   // uniform
        const float* lb = dL + (size_t)tb * E;
#pragma unroll
        for (int i = 0; i < XI; ++i)
#pragma unroll
            for (int g = 0; g < NX; ++g) xr[i][g] = xt[xo[i] + g];
#pragma unroll
        for (int j = 0; j < 8; ++j) br[j] = lb[bo[j]];
    };
    auto stage = [&](int buf, int tb, u32x4 (&xr)[XI][NX], float (&br)[8]) {
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            const int tl = lt + 2048 / CT * i;
            const int off = (lc >> 1) * kTile + tl * 32 + (lc & 1) * 16;
            if (tb + 32 > t1) {
#pragma unroll
                for (int g = 0; g < NX; ++g)
                    xr[i][g] = min(tb, last) + tl >= tb && tl < nrow ? xr[i][g] : (u32x4){0u, 0u, 0u, 0u};
            }
            if constexpr (BF) {
                *reinterpret_cast<u32x4*>(&s_x[buf][0][off]) = xr[i][0];
            } else {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(xr[i][j / 4][j % 4]);
                bf16x8 o[3];
                split3(v, o);
#pragma unroll
                for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8*>(&s_x[buf][p][off]) = o[p];
            }
        }
        if (wave < NT) {
            bf16x8 o[3];
            if (tb + 32 > t1) {
#pragma unroll
                for (int j = 0; j < 8; ++j) br[j] = min(tb, last) + 8 * q + j >= tb && 8 * q + j < nrow ? br[j] : 0.f;
            }
            split3(br, o);
#pragma unroll
            for (int p = 0; p < 3; ++p) s_b[buf][wave][p][lane] = __builtin_bit_cast(u32x4, o[p]);
        }
    };

#pragma unroll
    for (int u = 0; u < PD; ++u) load(t0 + 32 * u, xr[u], br[u]);
    auto tile = [&](int tb, int u) {
        const int buf = u & 1;
        stage(buf, tb, xr[u], br[u]);
        __syncthreads();   // also: every wave has left the buffer that is written next
        load(tb + 32 * PD, xr[u], br[u]);
        bf16x8 b[NW][3];
#pragma unroll
        for (int nt = 0; nt < NW; ++nt)
#pragma unroll
            for (int p = 0; p < 3; ++p) b[nt][p] = __builtin_bit_cast(bf16x8, s_b[buf][wn + nt][p][lane]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            bf16x8 a[TA];
#pragma unroll
            for (int p = 0; p < TA; ++p) {
                const __attribute__((address_space(3))) char* base =
                    (const __attribute__((address_space(3))) char*)(const __attribute__((address_space(3))) void*)
                        &s_x[buf][p][(wm + mt) * kTile];
                const uint32_t off = (uint32_t)(8 * q + m / 4) * 32u + (uint32_t)(m % 4) * 8u;
                const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(base + off));
                const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(base + off + 128u));
                a[p] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            }
#pragma unroll
            for (int nt = 0; nt < NW; ++nt) acc[mt][nt] = mfma_terms<TA, 3>(a, b[nt], acc[mt][nt]);
        }
    };
    for (int tb = t0; tb < t1; tb += 32 * PD) {
#pragma unroll
        for (int u = 0; u < PD; ++u)
            tile(tb + 32 * u, u);   // past the range: nothing but zeros
    }
    float* dst = part + (size_t)blockIdx.z * d * E;
    uint32_t again = 0;   // blocks with a NaN sum
#pragma unroll
    for (int nt = 0; nt < NW; ++nt) {
        const int e = e0 + 16 * (wn + nt) + m;
        if (e >= E) continue;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int c = c0 + 16 * (wm + mt) + 4 * q;
            if (c >= d) continue;   // d % 64 == 0: whole blocks
            const float sum[4] = {acc[mt][nt][0], acc[mt][nt][1], acc[mt][nt][2], acc[mt][nt][3]};
            if (any_nan(sum)) again |= 1u << (nt * MT + mt);
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[(size_t)(c + i) * E + e] = sum[i];
        }
    }
    while (again != 0) {   // in float32 from the operands, over what was written
        const int b = __ffs((int)again) - 1, e = e0 + 16 * (wn + b / MT) + m, c = c0 + 16 * (wm + b % MT) + 4 * q;
        again &= again - 1;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int t = t0; t < t1; ++t) {
            const float g = dL[(size_t)t * E + e];
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = fmaf(g, value_at<BF>(x, (size_t)t * d + c + i), sum[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[(size_t)(c + i) * E + e] = sum[i];
    }
}

// dw[i] = sum over the S token ranges of part[.][i], in order.
__global__ __launch_bounds__(256) void router_dw_reduce_kernel(const float* __restrict__ part, int S, size_t n,
                                                               float* __restrict__ dw) {
    constexpr int kB = 32;   // a latency or two for all ranges
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) {
        float s = 0.f;
        for (int b = 0; b < S; b += kB) {
            float v[kB];
#pragma unroll
            for (int u = 0; u < kB; ++u) v[u] = b + u < S ? part[(size_t)(b + u) * n + i] : 0.f;
#pragma unroll
            for (int u = 0; u < kB; ++u) s += v[u];
        }
        dw[i] = s;
    }
}

namespace {

// Expert blocks per workgroup, and the tokens of a range: ranges so that about
// two workgroups run on every compute unit, at least 128 tokens each.
struct RouterDwPlan {
    int nt, ct, wx, wy, rows, S;
};

RouterDwPlan router_dw_plan(int act, int T, int d, int E) {
    RouterDwPlan p{};
    p.nt = E <= 16 ? 1 : (E <= 32 ? 2 : 4);
    p.ct = act == kF32 ? 128 : 256;   // three x terms take the LDS of a wider tile
    p.wx = (d + p.ct - 1) / p.ct;
    p.wy = (E + 16 * p.nt - 1) / (16 * p.nt);
    const int want = std::max(1, 512 / (p.wx * p.wy));
    const int ranges = std::max(1, std::min(want, (T + 127) / 128));
    p.rows = ((T + ranges - 1) / ranges + 63) / 64 * 64;
    p.S = (T + p.rows - 1) / p.rows;
    return p;
}

template <bool BF>
void launch_router_dw_t(const float* dL, const void* x, float* dst, const RouterDwPlan& p, int T, int d, int E,
                        hipStream_t s) {
    constexpr int CT = BF ? 256 : 128;
    const dim3 g(p.wx, p.wy, p.S), b(256);
    if (p.nt == 1) hipLaunchKernelGGL((router_dw_kernel<BF, 1, CT>), g, b, 0, s, dL, x, dst, T, d, E, p.rows);
    else if (p.nt == 2) hipLaunchKernelGGL((router_dw_kernel<BF, 2, CT>), g, b, 0, s, dL, x, dst, T, d, E, p.rows);
    else hipLaunchKernelGGL((router_dw_kernel<BF, 4, CT>), g, b, 0, s, dL, x, dst, T, d, E, p.rows);
}

}  // namespace

// Workgroups of the resident kernel: two rounds of the two that a compute unit
// holds (T = 16384, d = 4096, E = 64 and T = 8192, d = 2048, E = 8: 512 of them
// 56 and 21 us, 1024 55 and 17, 2048 59 and 17).
constexpr int kDxGroups = 1024;

hipError_t launch_router_dx(int act, const float* dL, const void* w_router, const void* add, const int32_t* pos, int k,
                            void* dx, int T, int d, int E, hipStream_t s) {
    const int ncb = (d + 255) / 256;
    if (act != kF32 && !pos && E <= 64) {
        const int ranges = std::max(1, kDxGroups / ncb), rows = std::max(1, ((T + ranges - 1) / ranges + 63) / 64) * 64;
        const dim3 g((T + rows - 1) / rows * ncb), b(256);
        const uint16_t* w = static_cast<const uint16_t*>(w_router);
        const u32x4* in = static_cast<const u32x4*>(add);
        u32x4* out = static_cast<u32x4*>(dx);
        const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, g, b, 0, s, dL, w, in, out, T, d, E, rows); };
        const bool nt = past_caches((size_t)T * d * 2);
        if (E <= 32) nt ? go(router_dx_resident_kernel<1, true>) : go(router_dx_resident_kernel<1, false>);
        else nt ? go(router_dx_resident_kernel<2, true>) : go(router_dx_resident_kernel<2, false>);
        return hipGetLastError();
    }
    const dim3 g((T + 63) / 64 * ncb), b(256);
    if (act == kF32)
        hipLaunchKernelGGL((router_dx_kernel<false>), g, b, 0, s, dL, w_router, add, pos, k, dx, T, d, E);
    else
        hipLaunchKernelGGL((router_dx_kernel<true>), g, b, 0, s, dL, w_router, add, pos, k, dx, T, d, E);
    return hipGetLastError();
}

size_t router_dw_part_bytes(int act, int T, int d, int E) {
    const RouterDwPlan p = router_dw_plan(act, T, d, E);
    return p.S > 1 ? (size_t)p.S * d * E * 4 : 0;
}

hipError_t launch_router_dw(int act, const float* dL, const void* x, float* part, float* dw_router, int T, int d,
                            int E, hipStream_t s) {
    const RouterDwPlan p = router_dw_plan(act, T, d, E);
    float* dst = p.S > 1 ? part : dw_router;   // one range: no partial sums
    if (act == kF32) launch_router_dw_t<false>(dL, x, dst, p, T, d, E, s);
    else launch_router_dw_t<true>(dL, x, dst, p, T, d, E, s);
    if (p.S > 1) {
        const size_t n = (size_t)d * E;
        hipLaunchKernelGGL(router_dw_reduce_kernel, dim3((unsigned)std::min<size_t>((n + 255) / 256, 4096)), dim3(256),
                           0, s, part, p.S, n, dw_router);
    }
    return hipGetLastError();
}

}  // namespace moe
