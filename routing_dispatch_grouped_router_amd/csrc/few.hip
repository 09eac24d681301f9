// The routed block for a few tokens on the packed weights of moe_pack_weights, for
// gfx950: from router logits to y in three launches, four where the selection takes
// one of its own.  Given logits need no router: two or three.  Expert counts that are
// no multiple of 8 (float32: 4) have moe_route's router, which for bf16 rows
// transposes W_r first: up to five.
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
//
// The weights' bytes bound it.  d = 4096, E = 64, k = 8, H = 1536, bf16, one token:
// 61 us (302 MB, 4.9 TB/s; the up projection alone 36 us, 5.6 TB/s, as fast as a
// kernel that only reads); 16 tokens, d = 2048, E = 8, k = 4, H = 1024: 32 us (101 MB,
// 3.1 TB/s, of which router and selection 5 us and the launches' starts and ends
// 6); 7 tokens, two of them padding, of 128 MXFP8 experts, k = 4: 39 us (120 MB).  A
// 2 GiB copy runs at 4.9 TB/s on the same card.
#include <algorithm>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kRows = kFewTokens * kMaxTopK;
// Most logits that the up projection selects from itself.  One token of 64 experts: 62.1 us against 63.9 with a launch
// of its own, of 128 MXFP8 experts 20.1 and 20.7; 4 tokens of 64 experts 77.7 and 72.8 (4096 workgroups, each of which
// would select), one of 256 experts 24.6 and 22.6.
constexpr int kFused = 128;
constexpr int kFewSlice = 2048;   // most rows of W_r a workgroup of the router takes

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int wave_index() { return uniform((int)(threadIdx.x >> 6)); }

// ----------------------------------------------------------------------------- router

// Orderable image of a logit (larger logits larger, -0.0 as +0.0).
__device__ __forceinline__ uint32_t logit_key(float x) {
    uint32_t u = __float_as_uint(x);
    if (u == 0x80000000u) u = 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Partial logits of a token over a sixteenth of d, a workgroup each: part [T][16][E].
// W_r's rows are E / NV pieces of 16 bytes (C of them) and lie one after the
// other, so the workgroup's first 256 / C * C threads read consecutive pieces
// and keep their column.
template <bool BF>
__global__ __launch_bounds__(256) void few_logits_kernel(const u32x4* __restrict__ x, const u32x4* __restrict__ w,
                                                         float* __restrict__ part, int E, int d) {
    constexpr int NV = BF ? 8 : 4;
    constexpr int kB = 8;
    __shared__ float s_x[kFewSlice];
    __shared__ float red[256 * NV];
    const int t = blockIdx.y, tid = threadIdx.x, rows = d / kFewSlices, C = E / NV;
    const int by = 256 / C, n = rows * C;          // rows of a step; pieces of the slice
    const u32x4* wp = w + (size_t)blockIdx.x * n;
    const bool on = tid < by * C;
    u32x4 r[kB];
    auto request = [&](int p0) {
#pragma unroll
        for (int u = 0; u < kB; ++u) r[u] = wp[min(p0 + u * by * C + tid, n - 1)];
    };
    request(0);
    for (int c = tid; c < rows / NV + 1; c += 256) {   // d / 16 is a multiple of 4: the last piece may be half another's
        const size_t first = ((size_t)t * d + (size_t)blockIdx.x * rows) / NV;
        const int off = (int)(((size_t)t * d + (size_t)blockIdx.x * rows) % NV);
        if (NV * c - off >= rows) continue;
        float v[8];
        unpack16<BF>(x[first + c], v);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (NV * c + i >= off && NV * c + i - off < rows) s_x[NV * c + i - off] = v[i];
    }
    __syncthreads();
    float acc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = 0.f;
    for (int p0 = 0; p0 < n; p0 += kB * by * C) {
        if (p0) request(p0);
#pragma unroll
        for (int u = 0; u < kB; ++u) {
            const int p = p0 + u * by * C + tid;
            if (!on || p >= n) continue;
            float v[8];
            unpack16<BF>(r[u], v);
            const float xv = s_x[p / C];
#pragma unroll
            for (int i = 0; i < NV; ++i) acc[i] = fmaf(xv, v[i], acc[i]);
        }
    }
    // red [by][E]; the rows in order, 256 / E (at least one) ranges of them by a thread each, then the ranges
    if (on) {
#pragma unroll
        for (int i = 0; i < NV; ++i) red[NV * tid + i] = acc[i];
    }
    __syncthreads();
    const int ranges = min(by, max(1, 256 / E)), len = (by + ranges - 1) / ranges;
    for (int e = tid; e < E * ranges; e += 256) {
        const int g = e / E;
        float s = 0.f;
        for (int j = g * len; j < min(by, (g + 1) * len); ++j) s += red[j * E + e % E];
        acc[0] = s;   // E ranges > 256 only with one range: then the sum is the result
        if (ranges == 1) part[((size_t)t * kFewSlices + blockIdx.x) * E + e] = s;
    }
    if (ranges == 1) return;
    __syncthreads();
    if (tid < E * ranges) red[tid] = acc[0];
    __syncthreads();
    if (tid < E) {
        float s = red[tid];
        for (int g = 1; g < ranges; ++g) s += red[g * E + tid];
        part[((size_t)t * kFewSlices + blockIdx.x) * E + tid] = s;
    }
}

// The logit of a token and expert from its sixteen parts, in order.
__device__ __forceinline__ float join_parts(const float* part, int t, int e, int E) {
    const float* p = part + (size_t)t * kFewSlices * E + e;
    float v[kFewSlices];
#pragma unroll
    for (int i = 0; i < kFewSlices; ++i) v[i] = p[(size_t)i * E];
    float s = v[0];
#pragma unroll
    for (int i = 1; i < kFewSlices; ++i) s += v[i];
    return s;
}

// Gate j of the k selected logits, largest first.
__device__ __forceinline__ float gate_of(const float* val, int k, int j) {
    float sum = 0.f;
    for (int i = 0; i < k; ++i) sum += expf(val[i] - val[0]);
    return expf(val[j] - val[0]) / sum;
}

// A workgroup per token: logits from their sixteen parts (NULL: they are given),
// selection, gates.  An expert's rank is the number of experts before it,
// counted by 1024 / E threads each.
__global__ __launch_bounds__(1024) void few_select_kernel(const float* __restrict__ part, float* __restrict__ logits,
                                                          const uint8_t* __restrict__ mask, int32_t* __restrict__ idx,
                                                          float* __restrict__ gate, int E, int k) {
    __shared__ float s_logit[kMaxExperts];
    __shared__ int32_t s_rank[kMaxExperts];
    __shared__ float s_val[kMaxTopK];
    __shared__ int32_t s_idx[kMaxTopK];
    const int t = blockIdx.x, tid = threadIdx.x;
    if (tid < E) {
        float s;
        if (part) {
            s = join_parts(part, t, tid, E);
            logits[(size_t)t * E + tid] = s;
        } else {
            s = logits[(size_t)t * E + tid];
        }
        s_logit[tid] = s;
        s_rank[tid] = 0;
    }
    if (mask && mask[t] == 0) {
        if (tid < k) {
            idx[t * k + tid] = -1;
            gate[t * k + tid] = 0.f;
        }
        return;
    }
    __syncthreads();
    const int parts = 1024 / E, e = tid % E, mine_part = tid / E;
    if (mine_part < parts) {
        const uint32_t mine = logit_key(s_logit[e]);
        int before = 0;
        for (int o = mine_part; o < E; o += parts) {
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
        idx[t * k + tid] = s_idx[tid];
        gate[t * k + tid] = gate_of(s_val, k, tid);
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

// A uniform address plus a lane's 32-bit offset (an expert's weights and an
// activation buffer are below 2^32 bytes).
__device__ __forceinline__ u32x4 load16(const uint8_t* base, uint32_t off) {
    return *reinterpret_cast<const u32x4*>(base + off);
}

__device__ __forceinline__ int lane_row() { return (threadIdx.x & 15) >> 2; }                              // a, or t
__device__ __forceinline__ int lane_piece() { return 4 * ((threadIdx.x & 63) >> 4) + (threadIdx.x & 3); }   // p

// Weights [experts][rows][K] (scales [experts][K / 128][rows][4]) as a lane reads them: piece p of weight row
// row0 + 4 b + a of NB groups of 4 rows, `apart` rows from one group to the next.
template <int ACT>
struct Weights {
    const uint8_t* w;       // of the expert
    const uint8_t* s;
    uint32_t wo, so;        // the lane's offsets in group 0
};
template <int ACT>
constexpr int kWBytes = ACT == kF32 ? 4 : (ACT == kBF16 ? 2 : 1);

template <int ACT>
__device__ __forceinline__ Weights<ACT> weights_at(const uint8_t* w, const uint8_t* s, int e, int row0, int rows, int K) {
    const size_t expert = (size_t)e * rows * K;
    Weights<ACT> o;
    o.w = w + expert * kWBytes<ACT>;
    o.s = s + expert / 32;
    o.wo = (uint32_t)(row0 + lane_row()) * (uint32_t)(K * kWBytes<ACT>) + 16 * lane_piece();
    // piece p: elements 16 p .. of 256, scale (p / 2) % 4 of slice p / 8
    o.so = ACT == kMXFP8 ? (uint32_t)(((lane_piece() >> 3) * rows + row0 + lane_row()) * 4 + ((lane_piece() >> 1) & 3)) : 0u;
    return o;
}

// Offsets of rows rows[n0 ..] (n in all) of activations [.][TERMS][K], row r's line r / div; columns past the last row
// repeat it.
template <int ACT, int NT, int TERMS>
struct Acts {
    uint32_t x[NT];
};
template <int ACT, int NT, int TERMS>
__device__ __forceinline__ Acts<ACT, NT, TERMS> acts_at(const uint16_t* rows, int n0, int n, int div, int K) {
    Acts<ACT, NT, TERMS> o;
    const uint32_t term = (uint32_t)K * (ACT == kF32 ? 4u : 2u);
#pragma unroll
    for (int g = 0; g < NT; ++g)
        o.x[g] = (uint32_t)(rows[min(n0 + 4 * g + lane_row(), n - 1)] / div) * (TERMS * term) + (Seg<ACT>::kXBytes / 16) * lane_piece();
    return o;
}

// Whether a lane's piece of segment s is within K: the last segment may be half of one, the rest of it is zero.
template <int ACT>
__device__ __forceinline__ bool inside(int s, int K) {
    return (s + 1) * Seg<ACT>::kElems <= K || (threadIdx.x & 63) < 32;
}

// Segment s of the weights.  rows, K: theirs; group b is `step(b)` rows from the first.
template <int ACT, int NB, typename Step>
__device__ __forceinline__ void load_weights(const Weights<ACT>& p, int s, int rows, int K, Step step,
                                             WeightPiece<ACT, NB>& w) {
    if (inside<ACT>(s, K)) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            w.w[b] = load16(p.w + (size_t)step(b) * (K * kWBytes<ACT>) + 256 * (size_t)s, p.wo);
            if (ACT == kMXFP8) w.sc[b] = (p.s + (size_t)(2 * s) * rows * 4 + 4 * step(b))[p.so];
        }
    } else {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            w.w[b] = (u32x4){0u, 0u, 0u, 0u};
            w.sc[b] = 127u;
        }
    }
}

// Segment s of the activations.
template <int ACT, int NT, int TERMS>
__device__ __forceinline__ void load_acts(const uint8_t* x, const Acts<ACT, NT, TERMS>& in, int s, int K,
                                          ActPiece<ACT, NT, TERMS>& o) {
    const uint32_t term = (uint32_t)K * (ACT == kF32 ? 4u : 2u);
    if (inside<ACT>(s, K)) {
#pragma unroll
        for (int g = 0; g < NT; ++g)
#pragma unroll
            for (int t = 0; t < TERMS; ++t)
#pragma unroll
                for (int i = 0; i < Seg<ACT>::kX; ++i)
                    o.x[g][t][i] = load16(x + t * (size_t)term + (size_t)(Seg<ACT>::kXBytes * s + 16 * i), in.x[g]);
    } else {
#pragma unroll
        for (int g = 0; g < NT; ++g)
#pragma unroll
            for (int t = 0; t < TERMS; ++t)
#pragma unroll
                for (int i = 0; i < Seg<ACT>::kX; ++i) o.x[g][t][i] = (u32x4){0u, 0u, 0u, 0u};
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

template <int NB, int NT>
__device__ __forceinline__ void clear(f32x4 (&acc)[NB][NT]) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int g = 0; g < NT; ++g) acc[b][g] = (f32x4){0.f, 0.f, 0.f, 0.f};
}

// The wanted product of an accumulator: of weight row lane / 16 and activation row (lane % 16) / 4, the same on the
// four lanes of a quad.
__device__ __forceinline__ float wanted(const f32x4& v) {
    const int b = threadIdx.x & 3;
    const float mine = b & 2 ? (b & 1 ? v[3] : v[2]) : (b & 1 ? v[1] : v[0]);
    return __uint_as_float(group_reduce<4>(__float_as_uint(mine), AddF32()));
}

// The routed rows of group g, as a workgroup of 256 finds them in idx: with R <= E
// a group per routed row, whose rows are those of its expert if it is the
// expert's first row (none otherwise), else a group per expert.
template <typename Idx>
__device__ __forceinline__ int group_rows(const Idx& idx, int R, int E, int g, int& expert, uint16_t* rows, int32_t* cnt) {
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

// The rows of every expert in use as the down projection takes them: items of up to `most` rows of an expert each, in
// any order (it does not matter to any sum), rows[item_first ..] those rows.
struct FewList {
    int32_t items, pad[3];
    uint32_t item[kRows];    // expert, first row in rows, rows
    uint16_t rows[kRows];
};
static_assert(sizeof(FewList) == kFewListBytes, "its place in the workspace");
__device__ __forceinline__ int item_expert(uint32_t it) { return it >> 16; }
__device__ __forceinline__ int item_first(uint32_t it) { return (it >> 6) & 0x3FF; }
__device__ __forceinline__ int item_rows(uint32_t it) { return it & 0x3F; }

// A workgroup of 256 writes the list.
template <typename Idx>
__device__ __forceinline__ void make_list(const Idx& idx, int R, int E, int most, FewList* list) {
    __shared__ int32_t s_count[kMaxExperts], s_first[kMaxExperts];
    __shared__ int32_t s_items, s_total;
    const int tid = threadIdx.x;
    for (int e = tid; e < E; e += 256) s_count[e] = 0;
    if (tid == 0) s_items = s_total = 0;
    __syncthreads();
    int mine[2], slot[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = tid + 256 * i;
        mine[i] = r < R ? idx[r] : -1;
        slot[i] = mine[i] >= 0 && mine[i] < E ? atomicAdd(&s_count[mine[i]], 1) : -1;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (slot[i] == 0) {
            const int n = s_count[mine[i]], first = atomicAdd(&s_total, n), m = (n + most - 1) / most;
            s_first[mine[i]] = first;
            const int at = atomicAdd(&s_items, m);
            for (int j = 0; j < m; ++j)
                list->item[at + j] = (uint32_t)mine[i] << 16 | (uint32_t)(first + most * j) << 6 | (uint32_t)min(most, n - most * j);
        }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (slot[i] >= 0) list->rows[s_first[mine[i]] + slot[i]] = (uint16_t)(tid + 256 * i);
    if (tid == 0) list->items = s_items;
}

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
// of 4 gate rows and as many up; its waves take the quarters of K, D segments of
// it requested ahead.  SELECT (T E <= kFused, 256 / (T E) threads for each
// logit): every workgroup makes the selection for itself.  The first writes
// down the selection and the down projection's list (a workgroup of its own for
// that comes before one that no longer fits beside the others: 16 tokens of 8
// experts 34.5 us instead of 33.7, before what follows).
// Four waves a SIMD, so 128 registers, where it would take up to 190: more waves
// serve better than more loads ahead (bf16, d = 2048, 8 experts, H = 4096: 32 tokens 141
// -> 134 us, 20 tokens 103 -> 100.5; MXFP8, 64 experts, 32 tokens: 111 -> 104).  Five
// are slower; with 4 rows a reading it takes 76 to 88, and fewer cost more.
template <int ACT, int NB, int NT, int D, bool SELECT>
__global__ __launch_bounds__(256, NT == 1 ? 1 : 4) void few_up_kernel(const uint8_t* __restrict__ x, int32_t* __restrict__ idx,
                                                     float* __restrict__ gate, const float* __restrict__ part,
                                                     float* __restrict__ logits, const uint8_t* __restrict__ mask,
                                                     const uint8_t* __restrict__ w1, const uint8_t* __restrict__ s1,
                                                     void* __restrict__ h, FewList* __restrict__ list, int R, int E,
                                                     int k, int d, int H) {
    __shared__ uint16_t s_rows[kRows];
    __shared__ int32_t s_cnt[8];
    __shared__ float red[4][NB][NT][16];
    constexpr int units = 2 * NB;
    const bool lists = blockIdx.x == 0;
    const int nb = H / units, g = blockIdx.x / nb, hb = blockIdx.x - g * nb;
    int e, n;
    if constexpr (SELECT) {
        __shared__ float s_logit[kFused], s_val[kFused];
        __shared__ int32_t s_idx[kFused];
        __shared__ int32_t s_rank[kFused];
        const int N = R / k * E, tid = threadIdx.x;
        if (tid < N) {
            const float v = part ? join_parts(part, tid / E, tid % E, E) : logits[tid];
            s_logit[tid] = v;
            s_rank[tid] = 0;
            if (part && lists) logits[tid] = v;
        }
        __syncthreads();
        const int parts = 256 / N, at = tid % N, own = at % E, row = at - own;   // 256 / N threads count for each logit
        if (tid < parts * N) {
            const uint32_t key = logit_key(s_logit[at]);
            int before = 0;
#pragma unroll 8
            for (int o = tid / N; o < E; o += parts) {
                const uint32_t other = logit_key(s_logit[row + o]);
                before += other > key || (other == key && o < own);
            }
            atomicAdd(&s_rank[at], before);
        }
        __syncthreads();
        if (tid < N && s_rank[tid] < k) {
            const int t = tid / E;
            s_idx[t * k + s_rank[tid]] = mask && mask[t] == 0 ? -1 : own;
            s_val[t * k + s_rank[tid]] = s_logit[tid];
        }
        __syncthreads();
        if (lists) {
            if (tid < R) {
                idx[tid] = s_idx[tid];
                gate[tid] = s_idx[tid] < 0 ? 0.f : gate_of(s_val + tid / k * k, k, tid % k);
            }
            make_list(s_idx, R, E, 4 * NT, list);
        }
        n = group_rows(s_idx, R, E, g, e, s_rows, s_cnt);
    } else {
        if (lists) make_list(idx, R, E, 4 * NT, list);
        n = group_rows(idx, R, E, g, e, s_rows, s_cnt);
    }
    if (n == 0) return;
    const int u0 = units * hb, lane = threadIdx.x & 63, wave = wave_index();
    // packed rows of hidden unit u: gate at 64 (u / 32) + u % 32, up 32 further
    const Weights<ACT> p = weights_at<ACT>(w1, s1, e, 64 * (u0 / 32) + u0 % 32, 2 * H, d);
    auto step = [](int b) { return 4 * (b % (NB / 2)) + 32 * (b / (NB / 2)); };
    const int ns = (d + Seg<ACT>::kElems - 1) / Seg<ACT>::kElems, lo = wave * ns / 4, hi = (wave + 1) * ns / 4;
    for (int n0 = 0; n0 < n; n0 += 4 * NT) {
        const Acts<ACT, NT, 1> in = acts_at<ACT, NT, 1>(s_rows, n0, n, k, d);
        WeightPiece<ACT, NB> w[D];
        ActPiece<ACT, NT, 1> a[D];
        f32x4 acc[NB][NT];
        clear<NB, NT>(acc);
#pragma unroll
        for (int u = 0; u < D; ++u)
            if (lo + u < hi) {
                load_weights<ACT, NB>(p, lo + u, 2 * H, d, step, w[u]);
                load_acts<ACT, NT, 1>(x, in, lo + u, d, a[u]);
            }
        for (int s = lo; s < hi; s += D) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
                if (s + u >= hi) break;
                multiply<ACT, NB, NT, 1>(w[u], a[u], acc);
                if (s + u + D < hi) {
                    load_weights<ACT, NB>(p, s + u + D, 2 * H, d, step, w[u]);
                    load_acts<ACT, NT, 1>(x, in, s + u + D, d, a[u]);
                }
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float v = wanted(acc[b][t]);
                if ((lane & 3) == 0) red[wave][b][t][lane >> 2] = v;   // 4 (weight row) + row
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
// waves a quarter of K of one expert (up to 4 NT rows of it) in turn; the
// quarters of each routed row's outputs meet in LDS.  A quarter is a few segments,
// so a wave's requests run on over the ends of its experts: they are made by a
// cursor of their own, D segments ahead of the products.
template <int ACT, int NB, int NT, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void few_down_kernel(const uint8_t* __restrict__ h, const int32_t* __restrict__ idx,
                                                              const float* __restrict__ gate,
                                                              const FewList* __restrict__ list,
                                                              const uint8_t* __restrict__ w2,
                                                              const uint8_t* __restrict__ s2, void* __restrict__ y, int T,
                                                              int E, int k, int d, int H) {
    constexpr int TERMS = ACT == kF32 ? 1 : 2;
    constexpr int cols = 4 * NB, threads = 64 * WAVES;
    __shared__ uint32_t s_item[kRows];
    __shared__ uint16_t s_rows[kRows];
    __shared__ float s_gate[kRows];
    __shared__ uint8_t s_used[kRows];       // whether a slot is in use
    extern __shared__ float s_part[];   // [4][T k][cols]
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_index(), R = T * k;
    const int items = uniform(list->items);
    for (int r = tid; r < R; r += threads) {   // the list's ends are not written: read, not used
        s_item[r] = list->item[r];
        s_rows[r] = list->rows[r];
        s_gate[r] = gate[r];
        s_used[r] = idx[r] >= 0 && idx[r] < E;
    }
    __syncthreads();
    const int c0 = cols * blockIdx.x;
    const int ns = (H + Seg<ACT>::kElems - 1) / Seg<ACT>::kElems, quarter = wave & 3;
    const int lo = quarter * ns / 4, hi = (quarter + 1) * ns / 4;
    auto step = [](int b) { return 4 * b; };
    const int first_item = wave >> 2;
    if (lo < hi) {
        // the requests' cursor
        int gi = first_item, si = lo;
        Weights<ACT> p{};
        Acts<ACT, NT, TERMS> in{};
        auto enter = [&]() {
            if (gi >= items) return;
            const uint32_t it = uniform(s_item[gi]);
            p = weights_at<ACT>(w2, s2, item_expert(it), c0, d, H);
            in = acts_at<ACT, NT, TERMS>(s_rows + item_first(it), 0, item_rows(it), 1, H);
        };
        WeightPiece<ACT, NB> w[D];
        ActPiece<ACT, NT, TERMS> a[D];
        auto request = [&](int u) {
            if (gi >= items) return;
            load_weights<ACT, NB>(p, si, d, H, step, w[u]);
            load_acts<ACT, NT, TERMS>(h, in, si, H, a[u]);
            if (++si == hi) {
                si = lo;
                gi += WAVES / 4;
                enter();
            }
        };
        enter();
#pragma unroll
        for (int u = 0; u < D; ++u) request(u);
        f32x4 acc[NB][NT];
        clear<NB, NT>(acc);
        for (int g = first_item, s = lo; g < items;) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
                if (g >= items) break;
                multiply<ACT, NB, NT, TERMS>(w[u], a[u], acc);
                request(u);
                if (++s == hi) {
                    const uint32_t it = uniform(s_item[g]);
                    const uint16_t* rows = s_rows + item_first(it);
                    const int n = item_rows(it);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const int r = 4 * t + lane_row();
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const float v = wanted(acc[b][t]);
                            if ((lane & 3) == 0 && r < n)
                                s_part[((size_t)quarter * R + rows[r]) * cols + 4 * b + (lane >> 4)] = v;
                        }
                    }
                    clear<NB, NT>(acc);
                    s = lo;
                    g += WAVES / 4;
                }
            }
        }
    } else {   // a quarter without a segment
        for (int o = lane + 64 * first_item; o < R * cols; o += 16 * WAVES) s_part[(size_t)quarter * R * cols + o] = 0.f;
    }
    __syncthreads();
    for (int o = tid; o < T * cols; o += threads) {
        const int t = o / cols, c = o % cols;
        const float* q = s_part + (size_t)t * k * cols + c;
        const int by = R * cols;
        float s = 0.f;
#pragma unroll 4
        for (int j = 0; j < k; ++j, q += cols) {
            const float v = ((q[0] + q[by]) + q[2 * by]) + q[3 * by];   // of a slot not in use, what LDS held
            s = s_used[t * k + j] ? fmaf(s_gate[t * k + j], v, s) : s;
        }
        if (ACT == kF32) static_cast<float*>(y)[(size_t)t * d + c0 + c] = s;
        else static_cast<uint16_t*>(y)[(size_t)t * d + c0 + c] = f32_to_bf16(s);
    }
}

namespace {

// What the router left for the products: choices (or, `fused`, what they are made of) and where they go.
struct Choices {
    bool fused;
    const float* part;
    float* logits;
    const uint8_t* mask;
    int32_t* idx;
    float* gate;
    FewList* list;
};

template <int ACT, int NT>
hipError_t launch_products(const void* x_, const Choices& c, const uint8_t* w1, const uint8_t* w2, const uint8_t* s1,
                           const uint8_t* s2, void* h_, void* y, int T, int d, int E, int k, int H, hipStream_t s) {
    const int R = T * k, G = std::min(R, E);
    const uint8_t *x = static_cast<const uint8_t*>(x_), *h = static_cast<const uint8_t*>(h_);
    const dim3 up(G * (H / 8));
    if (c.fused)
        hipLaunchKernelGGL((few_up_kernel<ACT, 4, NT, 1, true>), up, dim3(256), 0, s, x, c.idx, c.gate, c.part, c.logits,
                           c.mask, w1, s1, h_, c.list, R, E, k, d, H);
    else
        hipLaunchKernelGGL((few_up_kernel<ACT, 4, NT, 1, false>), up, dim3(256), 0, s, x, c.idx, nullptr, nullptr, nullptr,
                           nullptr, w1, s1, h_, c.list, R, E, k, d, H);
    constexpr int D = NT == 1 ? 3 : 2;
    // LDS for the quarters of all rows: 32 KB at most
    if (R <= 256)
        hipLaunchKernelGGL((few_down_kernel<ACT, 2, NT, D, 8>), dim3(d / 8), dim3(512), (size_t)R * 128, s, h, c.idx,
                           c.gate, c.list, w2, s2, y, T, E, k, d, H);
    else
        hipLaunchKernelGGL((few_down_kernel<ACT, 1, NT, D, 8>), dim3(d / 4), dim3(512), (size_t)R * 64, s, h, c.idx,
                           c.gate, c.list, w2, s2, y, T, E, k, d, H);
    return hipGetLastError();
}

// Activation rows that a reading of the weights serves: 4 NT.  More of them cost
// loads and registers whether an expert has them or not; fewer a second reading,
// from the caches, where an expert has more.  bf16, d = 2048, by the rows that an
// expert has on average, us with 8 / 12 (/ 16) rows a reading:
//   5: E = 8, H = 1024 29.5 / 30.8;  6: E = 32, H = 1024 89.4 / 89.1, E = 8, H = 4096 87.4 / 89.7
//   7: E = 8, H = 1024 32.9 / 31.9;  8: E = 8, H = 1024 33.8 / 32.4, E = 32, H = 1024 103.9 / 93.1
//   10, 12 / 16: E = 8, H = 4096 100.5 / 106, H = 1024 36.7 / 37.8;  12: H = 4096 115.8 / 108.8, H = 1024 40.0 / 40.5.
// Float32 and MXFP8 weights take 8 at most: the second reading costs less than
// the registers (10 rows an expert: MXFP8, E = 8, H = 4096 83.8 / 85, float32, d = 1024 173 / 181).
// The average counts tokens that are padding, and skewed routing gives one expert several
// readings in a row.  With Zipf-routed logits (exponent 1.2, the largest expert 16 to 32
// rows) the choice and the best of the others, us from cold with the launches: 32 tokens, MXFP8,
// E = 128, k = 4 117 / 118, E = 64, k = 8 135 / 140; bf16, E = 64, k = 8 189 / 193, E = 128, k = 4,
// H = 512 116 / 112; float32, d = 1024, E = 64, k = 4, H = 512 119 / 115; 16 tokens, bf16,
// d = 4096, E = 64, k = 8, H = 1536 347 / 329: 5 % off at most.
template <int ACT>
hipError_t launch_products(const void* x, const Choices& c, const uint8_t* w1, const uint8_t* w2, const uint8_t* s1,
                           const uint8_t* s2, void* h, void* y, int T, int d, int E, int k, int H, hipStream_t s) {
    const float rows = (float)T * k / E;   // of an expert, on average
    if (T <= 4 || rows <= 2.f) return launch_products<ACT, 1>(x, c, w1, w2, s1, s2, h, y, T, d, E, k, H, s);
    if constexpr (ACT == kBF16) {
        if (T > 12 && rows > 11.f) return launch_products<ACT, 4>(x, c, w1, w2, s1, s2, h, y, T, d, E, k, H, s);
        if (T > 8 && rows >= 7.f)
            return launch_products<ACT, 3>(x, c, w1, w2, s1, s2, h, y, T, d, E, k, H, s);
    }
    return launch_products<ACT, 2>(x, c, w1, w2, s1, s2, h, y, T, d, E, k, H, s);
}

}  // namespace

bool few_routes_itself(int act, int d, int E) {
    return E % (act == kF32 ? 4 : 8) == 0 && E <= 1024 && d <= kFewSlices * kFewSlice;
}

hipError_t launch_few(int act, const void* x, const void* w_router, bool learned, float* logits, float* part,
                      const uint8_t* mask, const uint8_t* w1, const uint8_t* w2, const uint8_t* s1, const uint8_t* s2,
                      void* y, int32_t* idx, float* gate, void* list, void* h, int T, int d, int E, int k, int H,
                      hipStream_t s) {
    const u32x4 *xv = static_cast<const u32x4*>(x), *wv = static_cast<const u32x4*>(w_router);
    if (learned && act != kF32)
        hipLaunchKernelGGL(few_logits_kernel<true>, dim3(kFewSlices, T), dim3(256), 0, s, xv, wv, part, E, d);
    else if (learned)
        hipLaunchKernelGGL(few_logits_kernel<false>, dim3(kFewSlices, T), dim3(256), 0, s, xv, wv, part, E, d);
    const Choices c{T * E <= kFused, learned ? part : nullptr, logits, mask, idx, gate, static_cast<FewList*>(list)};
    if (!c.fused)
        hipLaunchKernelGGL(few_select_kernel, dim3(T), dim3(1024), 0, s, c.part, logits, mask, idx, gate, E, k);
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess) return st;
    if (act == kF32) return launch_products<kF32>(x, c, w1, w2, s1, s2, h, y, T, d, E, k, H, s);
    if (act == kBF16) return launch_products<kBF16>(x, c, w1, w2, s1, s2, h, y, T, d, E, k, H, s);
    return launch_products<kMXFP8>(x, c, w1, w2, s1, s2, h, y, T, d, E, k, H, s);
}

}  // namespace moe
