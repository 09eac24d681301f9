// The routed block for a few tokens on the packed weights of moe_pack_weights, for
// gfx950: three launches, from router logits to y.
//
//   logits = x W_r, top-k and gates;  h[r] = silu(x[t] Wg) (x[t] Wu) for the
//   routed rows r = t k + j with expert e_r;  y[t] = sum_j g[t][j] h[t k + j] Wd.
//
// Reading the weights of the experts in use is nearly all of the work.  The tiles
// of the block's grouped GEMMs, made for thousands of rows, would hold a row or
// two each; here the weights are the streamed operand and pass straight from
// memory into the matrix instructions, read once for all rows of their expert
// (up to 16 at a time).
//
// The operand layout.  A load is best where consecutive lanes read consecutive
// bytes; an MFMA operand wants a row per lane.  So a 16 x 16 MFMA takes 4 weight
// rows instead of 16, each in four operand rows: operand row 4 a + b holds weight
// row a at the 16-byte pieces p = 4 q + b of a 256-byte segment of K (q: the
// lane's quarter of the wave), so that 4 lanes read 64 consecutive bytes and a
// wave 256 of each of 4 rows.  Column 4 t + b holds the pieces b of activation row
// t in the same way.  Of the 16 x 16 products those with equal b are wanted, a
// value of the accumulator per lane, summed over the four lanes b.  A quarter of
// the matrix rate is used; the weights' bytes need a thirtieth of it.
//   float32 rows: v_mfma_f32_16x16x4_f32 (64 of K a segment); bfloat16:
//   v_mfma_f32_16x16x32_bf16 (128 of K); MXFP8 weights: their codes times the block's
//   power of two are exact in bfloat16, x is bfloat16 (256 of K).
// h is float32 for float32 blocks, else two bfloat16 terms (2^-16 of it left out).
//
// Every sum over K is taken in four quarters, added in order, whatever the other
// rows are: a token's result does not depend on the tokens beside it.
#include <algorithm>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kRows = kFewTokens * kMaxTopK;

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int wave_index() { return uniform((int)(threadIdx.x >> 6)); }

// ----------------------------------------------------------------------------- router

// Orderable image of a logit (larger logits larger, -0.0 as +0.0).
__device__ __forceinline__ uint32_t logit_key(float x) {
    uint32_t u = __float_as_uint(x);
    if (u == 0x80000000u) u = 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// A workgroup per token: logits (LEARNED, E / NV a power of two up to 64, NV
// values a 16-byte load), selection, gates.  Wave w takes the w-th sixteenth of
// d, its lanes consecutive 16-byte pieces of W_r; an expert's rank is the number
// of experts before it, counted by 1024 / E threads each.
template <bool LEARNED, bool BF>
__global__ __launch_bounds__(1024) void few_route_kernel(const void* __restrict__ x, const void* __restrict__ w,
                                                         float* __restrict__ logits,
                                                         const uint8_t* __restrict__ mask, int32_t* __restrict__ idx,
                                                         float* __restrict__ gate, int E, int k, int d) {
    constexpr int NV = BF ? 8 : 4;
    __shared__ float s_logit[kMaxExperts];
    __shared__ int32_t s_rank[kMaxExperts];
    __shared__ float s_val[kMaxTopK];
    __shared__ int32_t s_idx[kMaxTopK];
    extern __shared__ float s_dyn[];   // x [d], then the waves' sums [16][E]
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = wave_index();
    if (LEARNED) {
        float* s_x = s_dyn;
        float* s_sum = s_dyn + d;
        for (int c = tid; c < d / NV; c += 1024) {
            float v[8];
            unpack16<BF>(static_cast<const u32x4*>(x)[(size_t)t * (d / NV) + c], v);
#pragma unroll
            for (int i = 0; i < NV; ++i) s_x[NV * c + i] = v[i];
        }
        __syncthreads();
        const int C = E / NV;                     // pieces of a row of W_r
        const int lo = wave * (d / 16), hi = lo + d / 16;
        const u32x4* wp = static_cast<const u32x4*>(w) + (size_t)lo * C;
        const int n = (hi - lo) * C, by = 64 / C;  // pieces of this wave's rows; rows of 64 of them
        float acc[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) acc[i] = 0.f;
        constexpr int kB = 8;
        for (int p = lane; p < n; p += 64 * kB) {
            u32x4 r[kB];
#pragma unroll
            for (int u = 0; u < kB; ++u) r[u] = wp[min(p + 64 * u, n - 1)];
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                if (p + 64 * u >= n) continue;
                float v[8];
                unpack16<BF>(r[u], v);
                const float xv = s_x[lo + p / C + by * u];
#pragma unroll
                for (int i = 0; i < NV; ++i) acc[i] = fmaf(xv, v[i], acc[i]);
            }
        }
        for (int m = C; m < 64; m <<= 1)
#pragma unroll
            for (int i = 0; i < NV; ++i) acc[i] += __shfl_xor(acc[i], m);
        if (lane < C) {
#pragma unroll
            for (int i = 0; i < NV; ++i) s_sum[wave * E + NV * lane + i] = acc[i];
        }
        __syncthreads();
        if (tid < E) {
            float s = s_sum[tid];
#pragma unroll
            for (int v = 1; v < 16; ++v) s += s_sum[v * E + tid];
            s_logit[tid] = s;
            logits[(size_t)t * E + tid] = s;
        }
    } else if (tid < E) {
        s_logit[tid] = logits[(size_t)t * E + tid];
    }
    if (mask && mask[t] == 0) {
        if (tid < k) {
            idx[t * k + tid] = -1;
            gate[t * k + tid] = 0.f;
        }
        return;
    }
    if (tid < E) s_rank[tid] = 0;
    __syncthreads();
    const int parts = 1024 / E, e = tid % E, part = tid / E;
    if (part < parts) {
        const uint32_t mine = logit_key(s_logit[e]);
        int before = 0;
        for (int o = part; o < E; o += parts) {
            const uint32_t other = logit_key(s_logit[o]);
            before += other > mine || (other == mine && o < e);
        }
        atomicAdd(&s_rank[e], before);
    }
    __syncthreads();
    if (tid < E && s_rank[tid] < k) {
        s_idx[s_rank[tid]] = tid;
        s_val[s_rank[tid]] = s_logit[tid];
    }
    __syncthreads();
    if (tid < k) {
        float sum = 0.f;
        for (int j = 0; j < k; ++j) sum += expf(s_val[j] - s_val[0]);
        idx[t * k + tid] = s_idx[tid];
        gate[t * k + tid] = expf(s_val[tid] - s_val[0]) / sum;
    }
}

// ----------------------------------------------------------------------------- the products

// ACT: kF32, kBF16 or kMXFP8 weights.
template <int ACT>
struct Seg {
    static constexpr int kXBytes = ACT == kMXFP8 ? 512 : 256;               // of an activation row
    static constexpr int kX = ACT == kMXFP8 ? 2 : 1;                        // 16-byte loads of a lane's piece of it
    static constexpr int kElems = ACT == kF32 ? 64 : (ACT == kBF16 ? 128 : 256);
};

template <int ACT, int NB>
struct WeightPiece {
    u32x4 w[NB];
    uint32_t sc[NB];     // MXFP8: the piece's scale
};
template <int ACT, int NT, int TERMS>
struct ActPiece {
    u32x4 x[NT][TERMS][Seg<ACT>::kX];
};

// NB groups of 4 weight rows, row0[b] + the lane's, of an expert's [rows][K].
template <int ACT, int NB>
struct Weights {
    const uint8_t* w[NB];
    const uint8_t* s[NB];   // scales [K / 128][rows][4]
    size_t slice;           // bytes of a 128-wide slice of them
    int K;
};

template <int ACT, int NB>
__device__ __forceinline__ Weights<ACT, NB> weights_at(const uint8_t* w, const uint8_t* s, const int (&row0)[NB], int rows,
                                                       int K) {
    const int lane = threadIdx.x & 63, a = (lane & 15) >> 2, p = 4 * (lane >> 4) + (lane & 3);
    const size_t pitch = (size_t)K * (ACT == kF32 ? 4 : (ACT == kBF16 ? 2 : 1));
    Weights<ACT, NB> o;
    o.slice = (size_t)rows * 4;
    o.K = K;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        o.w[b] = w + (size_t)(row0[b] + a) * pitch + 16 * p;
        // piece p: elements 16 p .. of 256, scale (p / 2) % 4 of slice p / 8
        o.s[b] = ACT == kMXFP8 ? s + (p >> 3) * o.slice + (size_t)(row0[b] + a) * 4 + ((p >> 1) & 3) : nullptr;
    }
    return o;
}

// Rows rows[n0 ..] (n in all) of activations x [.][TERMS][K], row r's line r / div; columns past the last row repeat it.
template <int ACT, int NT, int TERMS>
struct Acts {
    const uint8_t* x[NT];
    uint32_t term;
};
template <int ACT, int NT, int TERMS>
__device__ __forceinline__ Acts<ACT, NT, TERMS> acts_at(const void* x, const uint16_t* rows, int n0, int n, int div, int K) {
    const int lane = threadIdx.x & 63, t = (lane & 15) >> 2, p = 4 * (lane >> 4) + (lane & 3);
    Acts<ACT, NT, TERMS> o;
    o.term = (uint32_t)K * (ACT == kF32 ? 4u : 2u);
#pragma unroll
    for (int g = 0; g < NT; ++g) {
        const int line = rows[min(n0 + 4 * g + t, n - 1)] / div;
        o.x[g] = static_cast<const uint8_t*>(x) + (size_t)line * TERMS * o.term + (Seg<ACT>::kXBytes / 16) * p;
    }
    return o;
}

// Whether this lane's piece of segment s is inside K (the last segment may be half of one).
template <int ACT>
__device__ __forceinline__ bool inside(int s, int K) {
    return (s + 1) * Seg<ACT>::kElems <= K || (threadIdx.x & 63) < 32;
}

template <int ACT, int NB>
__device__ __forceinline__ void load(const Weights<ACT, NB>& p, int s, WeightPiece<ACT, NB>& o) {
    if (inside<ACT>(s, p.K)) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            o.w[b] = *reinterpret_cast<const u32x4*>(p.w[b] + 256 * (size_t)s);
            if (ACT == kMXFP8) o.sc[b] = p.s[b][2 * s * p.slice];
        }
    } else {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            o.w[b] = (u32x4){0u, 0u, 0u, 0u};
            o.sc[b] = 127u;
        }
    }
}
template <int ACT, int NT, int TERMS>
__device__ __forceinline__ void load(const Acts<ACT, NT, TERMS>& p, int s, int K, ActPiece<ACT, NT, TERMS>& o) {
    const bool in = inside<ACT>(s, K);
#pragma unroll
    for (int g = 0; g < NT; ++g)
#pragma unroll
        for (int t = 0; t < TERMS; ++t)
#pragma unroll
            for (int i = 0; i < Seg<ACT>::kX; ++i) {
                if (in) o.x[g][t][i] = *reinterpret_cast<const u32x4*>(p.x[g] + t * p.term + Seg<ACT>::kXBytes * s + 16 * i);
                else o.x[g][t][i] = (u32x4){0u, 0u, 0u, 0u};
            }
}

// Eight E4M3 codes times 2^(byte - 127) as bfloat16 (exact).
__device__ __forceinline__ bf16x8 fp8_to_bf16(uint32_t lo, uint32_t hi, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return (bf16x8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <int ACT, int NB, int NT, int TERMS>
__device__ __forceinline__ void multiply(const WeightPiece<ACT, NB>& w, const ActPiece<ACT, NT, TERMS>& x,
                                         f32x4 (&acc)[NB][NT]) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        if constexpr (ACT == kF32) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int g = 0; g < NT; ++g)
                    acc[b][g] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w.w[b][j]),
                                                                     __uint_as_float(x.x[g][0][0][j]), acc[b][g], 0, 0, 0);
        } else if constexpr (ACT == kBF16) {
            const bf16x8 wv = __builtin_bit_cast(bf16x8, w.w[b]);
#pragma unroll
            for (int t = 0; t < TERMS; ++t)
#pragma unroll
                for (int g = 0; g < NT; ++g)
                    acc[b][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, __builtin_bit_cast(bf16x8, x.x[g][t][0]),
                                                                        acc[b][g], 0, 0, 0);
        } else {
            const float scale = __uint_as_float(w.sc[b] << 23);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bf16x8 wv = fp8_to_bf16(w.w[b][2 * i], w.w[b][2 * i + 1], scale);
#pragma unroll
                for (int t = 0; t < TERMS; ++t)
#pragma unroll
                    for (int g = 0; g < NT; ++g)
                        acc[b][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            wv, __builtin_bit_cast(bf16x8, x.x[g][t][i]), acc[b][g], 0, 0, 0);
            }
        }
    }
}

// sum[b][g]: of weight row 4 b + lane / 16 and row 4 g + (lane % 16) / 4, the same on the four lanes of a quad: the
// product over the segments [s0, s1), D of them requested ahead.
template <int ACT, int NB, int NT, int TERMS, int D>
__device__ __forceinline__ void product(const Weights<ACT, NB>& p, const Acts<ACT, NT, TERMS>& in, int s0, int s1,
                                        float (&sum)[NB][NT]) {
    WeightPiece<ACT, NB> w[D];
    ActPiece<ACT, NT, TERMS> x[D];
    f32x4 acc[NB][NT];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int g = 0; g < NT; ++g) acc[b][g] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < D; ++u)
        if (s0 + u < s1) {
            load(p, s0 + u, w[u]);
            load(in, s0 + u, p.K, x[u]);
        }
    for (int s = s0; s < s1; s += D) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
            if (s + u >= s1) break;
            multiply<ACT, NB, NT, TERMS>(w[u], x[u], acc);
            if (s + u + D < s1) {
                load(p, s + u + D, w[u]);
                load(in, s + u + D, p.K, x[u]);
            }
        }
    }
    const int b4 = threadIdx.x & 3;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int g = 0; g < NT; ++g) {
            const f32x4 v = acc[b][g];
            const float mine = b4 & 2 ? (b4 & 1 ? v[3] : v[2]) : (b4 & 1 ? v[1] : v[0]);
            sum[b][g] = __uint_as_float(group_reduce<4>(__float_as_uint(mine), AddF32()));
        }
}

// The routed rows of group g, as a workgroup of 256 finds them in idx: with R <= E
// a group per routed row, whose rows are those of its expert if it is the
// expert's first row (none otherwise), else a group per expert.
__device__ __forceinline__ int group_rows(const int32_t* idx, int R, int E, int g, int& expert, uint16_t* rows, int32_t* cnt) {
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
    expert = R <= E ? uniform(idx[g]) : g;
    if (expert < 0 || expert >= E) return 0;
    const int r0 = tid, r1 = 256 + tid;
    const int v0 = r0 < R ? idx[r0] : -1, v1 = r1 < R ? idx[r1] : -1;
    const uint64_t b0 = __ballot(v0 == expert), b1 = __ballot(v1 == expert);
    if (lane == 0) {
        cnt[wave] = __popcll(b0);
        cnt[4 + wave] = __popcll(b1);
    }
    __syncthreads();
    int off0 = 0, off1 = 0, n = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        if (w == wave) off0 = n;
        if (w == 4 + wave) off1 = n;
        n += cnt[w];
    }
    const uint64_t below = (1ull << lane) - 1ull;
    if (v0 == expert) rows[off0 + __popcll(b0 & below)] = (uint16_t)r0;
    if (v1 == expert) rows[off1 + __popcll(b1 & below)] = (uint16_t)r1;
    __syncthreads();
    n = uniform(n);
    if (R <= E && uniform(rows[0]) != g) return 0;   // another row of this expert comes first
    return n;
}
static_assert(kRows <= 512, "two rows a thread");

// h of one hidden unit, stored as the down projection reads it.
template <int ACT>
__device__ __forceinline__ void store_h(float a, float b, void* h, size_t row, int H, int u) {
#pragma clang fp contract(off)
    const float o = a / (1.0f + expf(-a)) * b;
    if (ACT == kF32) {
        static_cast<float*>(h)[row * H + u] = o;
    } else {   // the first term ends at bfloat16's largest value: past it, the remainder of infinity would be NaN
        constexpr float kMax = 0x1.fep127f;
        const float hi = bf16_round(fminf(fmaxf(o, -kMax), kMax));
        uint16_t* p = static_cast<uint16_t*>(h) + row * 2 * H + u;
        p[0] = f32_to_bf16(hi);
        p[H] = f32_to_bf16(o - hi);
    }
}

}  // namespace

// Gate and up projections: workgroup = (group, 2 NB hidden units), NB / 2 groups
// of 4 gate rows and as many up; its waves take the quarters of K.
template <int ACT, int NB, int NT, int D>
__global__ __launch_bounds__(256) void few_up_kernel(const void* __restrict__ x, const int32_t* __restrict__ idx,
                                                     const uint8_t* __restrict__ w1, const uint8_t* __restrict__ s1,
                                                     void* __restrict__ h, int R, int E, int k, int d, int H) {
    __shared__ uint16_t s_rows[kRows];
    __shared__ int32_t s_cnt[8];
    __shared__ float red[4][NB][NT][16];
    constexpr int units = 2 * NB;
    const int nb = H / units, g = blockIdx.x / nb, hb = blockIdx.x - g * nb;
    int e;
    const int n = group_rows(idx, R, E, g, e, s_rows, s_cnt);
    if (n == 0) return;
    const int u0 = units * hb, lane = threadIdx.x & 63, wave = wave_index();
    // packed rows of hidden unit u: gate at 64 (u / 32) + u % 32, up 32 further
    int row0[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) row0[b] = 64 * (u0 / 32) + u0 % 32 + 4 * (b % (NB / 2)) + 32 * (b / (NB / 2));
    const size_t expert = (size_t)e * 2 * H * d;
    const Weights<ACT, NB> p = weights_at<ACT, NB>(w1 + expert * (ACT == kF32 ? 4 : (ACT == kBF16 ? 2 : 1)),
                                                   s1 + expert / 32, row0, 2 * H, d);
    const int ns = (d + Seg<ACT>::kElems - 1) / Seg<ACT>::kElems, lo = wave * ns / 4, hi = (wave + 1) * ns / 4;
    for (int n0 = 0; n0 < n; n0 += 4 * NT) {
        const Acts<ACT, NT, 1> in = acts_at<ACT, NT, 1>(x, s_rows, n0, n, k, d);
        float sum[NB][NT];
        product<ACT, NB, NT, 1, D>(p, in, lo, hi, sum);
        if ((lane & 3) == 0) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int t = 0; t < NT; ++t) red[wave][b][t][lane >> 2] = sum[b][t];   // 4 (weight row) + row
        }
        __syncthreads();
        for (int o = threadIdx.x; o < units * 4 * NT; o += 256) {
            const int u = o % units, r = o / units, at = 4 * (u & 3) + (r & 3);
            if (n0 + r < n) {
                auto total = [&](int b) {
                    return ((red[0][b][r >> 2][at] + red[1][b][r >> 2][at]) + red[2][b][r >> 2][at]) + red[3][b][r >> 2][at];
                };
                store_h<ACT>(total(u >> 2), total((u >> 2) + NB / 2), h, s_rows[n0 + r], H, u0 + u);
            }
        }
        if (n0 + 4 * NT < n) __syncthreads();
    }
}

// Down projection and combine: workgroup = 4 NB outputs of every token, its
// sixteen waves a quarter of K of one expert in turn; the quarters of each
// routed row's outputs meet in LDS.
template <int ACT, int NB, int NT, int D>
__global__ __launch_bounds__(1024) void few_down_kernel(const void* __restrict__ h, const int32_t* __restrict__ idx,
                                                        const float* __restrict__ gate,
                                                        const uint8_t* __restrict__ w2, const uint8_t* __restrict__ s2,
                                                        void* __restrict__ y, int T, int E, int k, int d, int H) {
    constexpr int TERMS = ACT == kF32 ? 1 : 2;
    constexpr int cols = 4 * NB;
    __shared__ int32_t s_count[kMaxExperts], s_first[kMaxExperts];
    __shared__ int32_t s_expert[kRows];
    __shared__ uint16_t s_rows[kRows];
    __shared__ int32_t s_groups, s_total;
    extern __shared__ float s_part[];   // [4][T k][cols]
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_index(), R = T * k;
    // the experts in use and their rows; their order does not matter to any sum
    for (int e = tid; e < E; e += 1024) s_count[e] = 0;
    if (tid == 0) s_groups = s_total = 0;
    __syncthreads();
    int mine = -1, slot = 0;
    if (tid < R) {
        mine = idx[tid];
        if (mine < 0 || mine >= E) mine = -1;
        else slot = atomicAdd(&s_count[mine], 1);
    }
    __syncthreads();
    if (mine >= 0 && slot == 0) {
        s_expert[atomicAdd(&s_groups, 1)] = mine;
        s_first[mine] = atomicAdd(&s_total, s_count[mine]);
    }
    __syncthreads();
    if (mine >= 0) s_rows[s_first[mine] + slot] = (uint16_t)tid;
    __syncthreads();
    const int c0 = cols * blockIdx.x, groups = uniform(s_groups);
    const int ns = (H + Seg<ACT>::kElems - 1) / Seg<ACT>::kElems, quarter = wave & 3;
    const int lo = quarter * ns / 4, hi = (quarter + 1) * ns / 4;
    int row0[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) row0[b] = c0 + 4 * b;
    for (int g = wave >> 2; g < groups; g += 4) {
        const int e = uniform(s_expert[g]), n = uniform(s_count[e]);
        const uint16_t* rows = s_rows + uniform(s_first[e]);
        const size_t expert = (size_t)e * d * H;
        const Weights<ACT, NB> p = weights_at<ACT, NB>(w2 + expert * (ACT == kF32 ? 4 : (ACT == kBF16 ? 2 : 1)),
                                                       s2 + expert / 32, row0, d, H);
        for (int n0 = 0; n0 < n; n0 += 4 * NT) {
            const Acts<ACT, NT, TERMS> in = acts_at<ACT, NT, TERMS>(h, rows, n0, n, 1, H);
            float sum[NB][NT];
            product<ACT, NB, NT, TERMS, D>(p, in, lo, hi, sum);
            if ((lane & 3) == 0) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int r = n0 + 4 * t + ((lane & 15) >> 2);
                    if (r < n) {
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            s_part[((size_t)quarter * R + rows[r]) * cols + 4 * b + (lane >> 4)] = sum[b][t];
                    }
                }
            }
        }
    }
    __syncthreads();
    for (int o = tid; o < T * cols; o += 1024) {
        const int t = o / cols, c = o % cols;
        float s = 0.f;
        for (int j = 0; j < k; ++j) {
            const int r = t * k + j, e = idx[r];
            if (e < 0 || e >= E) continue;
            const float* q = s_part + (size_t)r * cols + c;
            const size_t by = (size_t)R * cols;
            s = fmaf(gate[r], ((q[0] + q[by]) + q[2 * by]) + q[3 * by], s);
        }
        if (ACT == kF32) static_cast<float*>(y)[(size_t)t * d + c0 + c] = s;
        else static_cast<uint16_t*>(y)[(size_t)t * d + c0 + c] = f32_to_bf16(s);
    }
}

namespace {

template <int ACT>
hipError_t launch_products(const void* x, const int32_t* idx, const float* gate, const uint8_t* w1, const uint8_t* w2,
                           const uint8_t* s1, const uint8_t* s2, void* h, void* y, int T, int d, int E, int k, int H,
                           hipStream_t s) {
    const int R = T * k, G = std::min(R, E);
    hipLaunchKernelGGL((few_up_kernel<ACT, 4, 4, 1>), dim3(G * (H / 8)), dim3(256), 0, s, x, idx, w1, s1, h, R, E, k, d, H);
    // LDS for the quarters of all rows: 32 KB at most
    if (R <= 256)
        hipLaunchKernelGGL((few_down_kernel<ACT, 2, 4, 1>), dim3(d / 8), dim3(1024), (size_t)4 * R * 8 * 4, s, h, idx, gate, w2,
                           s2, y, T, E, k, d, H);
    else
        hipLaunchKernelGGL((few_down_kernel<ACT, 1, 4, 1>), dim3(d / 4), dim3(1024), (size_t)4 * R * 4 * 4, s, h, idx, gate, w2,
                           s2, y, T, E, k, d, H);
    return hipGetLastError();
}

}  // namespace

bool few_routes_itself(int act, int d, int E) {
    const int nv = act == kF32 ? 4 : 8, c = E / nv;
    return E % nv == 0 && c <= 64 && (c & (c - 1)) == 0 && 4 * d + 64 * E <= 48 * 1024;   // its LDS
}

hipError_t launch_few(int act, const void* x, const void* w_router, bool learned, float* logits, const uint8_t* mask,
                      const uint8_t* w1, const uint8_t* w2, const uint8_t* s1, const uint8_t* s2, void* y, int32_t* idx,
                      float* gate, void* h, int T, int d, int E, int k, int H, hipStream_t s) {
    const bool bf = act != kF32;
    const size_t lds = (size_t)(d + 16 * E) * 4;
    if (!learned)
        hipLaunchKernelGGL((few_route_kernel<false, true>), dim3(T), dim3(1024), 0, s, x, w_router, logits, mask, idx, gate, E, k, d);
    else if (bf)
        hipLaunchKernelGGL((few_route_kernel<true, true>), dim3(T), dim3(1024), lds, s, x, w_router, logits, mask, idx, gate, E, k, d);
    else
        hipLaunchKernelGGL((few_route_kernel<true, false>), dim3(T), dim3(1024), lds, s, x, w_router, logits, mask, idx, gate, E, k, d);
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess) return st;
    if (act == kF32) return launch_products<kF32>(x, idx, gate, w1, w2, s1, s2, h, y, T, d, E, k, H, s);
    if (act == kBF16) return launch_products<kBF16>(x, idx, gate, w1, w2, s1, s2, h, y, T, d, E, k, H, s);
    return launch_products<kMXFP8>(x, idx, gate, w1, w2, s1, s2, h, y, T, d, E, k, H, s);
}

}  // namespace moe
