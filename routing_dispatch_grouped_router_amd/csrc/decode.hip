// The experts of a few tokens with 4-bit weights, for gfx950 (serving: T from
// one token to kDecodeTokens).
//
// Weights are MXFP4 (OCP MX v1.0): E2M1 codes, two to a byte with the even
// element in the low four bits, and one E8M0 scale byte per 32 elements along
// the contraction axis; codes and scales are row-major:
//   W1 [E][2H][d/2] (rows as moe_pack_weights orders them: 32 gate, 32 up, ...),
//   W2 [E][d][H/2], S1 [E][2H][d/32], S2 [E][d][H/32].
// For the R = T k routed rows r = t k + j with expert e_r:
//   h[r] = silu(x[t] Wg) (x[t] Wu),  ye[r] = h[r] Wd,  y[t] = sum_j g[t][j] ye[t k + j].
// Reading the weights of the experts in use is nearly all of the work, so a
// group of rows of one expert reads each weight once: 16 weight rows are the M
// operand, up to 16 routed rows the N operand of v_mfma_f32_16x16x32_bf16.  An
// E2M1 value times a power of two is exact in bfloat16, so the weights are
// converted in registers (v_cvt_scalef32_pk_bf16_fp4) without a rounding, and
// the activations stay bfloat16.  Rows are not sorted or moved: a workgroup
// finds its expert's rows in topk_idx itself, and an index outside [0, E) is a
// slot not in use.
//
// Every sum over K is taken in four quarters (of K / 128 slices, in order) that
// are added in order, whichever kernel and however many rows: a token's result
// does not depend on the tokens beside it.
#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kMaxRows = kDecodeTokens * kMaxTopK;

// This wave's index, and a value that is the same on all its lanes, known to be
// uniform: the branches around the MFMAs (which ignore the lane mask) have to
// be scalar ones.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int wave_index() { return uniform((int)(threadIdx.x >> 6)); }

__device__ __forceinline__ float e8m0_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight E2M1 codes times 2^(byte - 127) as bfloat16 (exact).
__device__ __forceinline__ bf16x8 fp4_to_bf16(uint32_t w, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    return (bf16x8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Row list of a group: LDS for every routed row.
struct GroupRows {
    uint16_t rows[kMaxRows];
    int32_t cnt[4];
};

// The routed rows of group g: with R <= E a group per routed row, whose rows
// are those of its expert if it is the expert's first row (none otherwise);
// else a group per expert.  rows[0, n) in ascending order; returns n, the
// same on every thread of the workgroup's 256.
__device__ __forceinline__ int group_rows(const int32_t* idx, int R, int E, int g, int& expert, GroupRows& s) {
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
    if (R <= 64) {   // one load; every wave writes the same list and reads its own writes
        const int mine = lane < R ? idx[lane] : -1;
        expert = R <= E ? uniform(__shfl(mine, g)) : g;
        if (expert < 0 || expert >= E) return 0;
        const uint64_t b = __ballot(mine == expert);
        if (R <= E && __ffsll((unsigned long long)b) - 1 != g) return 0;   // another row of this expert comes first
        if (mine == expert) s.rows[__popcll(b & ((1ull << lane) - 1ull))] = (uint16_t)lane;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        return __popcll(b);
    }
    expert = R <= E ? uniform(idx[g]) : g;
    if (expert < 0 || expert >= E) return 0;
    int n = 0;
    for (int base = 0; base < R; base += 256) {
        const int r = base + tid;
        const bool mine = r < R && idx[r] == expert;
        const uint64_t b = __ballot(mine);
        if (lane == 0) s.cnt[wave] = __popcll(b);
        __syncthreads();
        int off = n, all = n;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w < wave) off += s.cnt[w];
            all += s.cnt[w];
        }
        if (mine) s.rows[off + __popcll(b & ((1ull << lane) - 1ull))] = (uint16_t)r;
        n = uniform(all);
        __syncthreads();   // cnt is rewritten by the next 256 rows; rows[] is complete after the last
    }
    if (R <= E && uniform(s.rows[0]) != g) return 0;   // another row of this expert comes first
    return n;
}

// What a wave streams: NB blocks of 16 weight rows against 16 routed rows.
// The memory pipe takes one access a clock for four consecutive lanes of one
// 64-byte piece, but for every lane of its own row if the lanes are laid out
// as the MFMA operands need them (rows across consecutive lanes: 390 accesses
// a slice, and the kernel ran at that pipe's rate, 2.7 TB/s).  So four lanes
// load 64 bytes of a weight row, sixteen 256 bytes of an activation row, and
// the operands are gathered through a wave-private LDS stage (no barrier: one
// wave writes and reads it, in order).
//   w : chunk c (16 bytes, one scale block) of row r at 4 r + (c + r / 4) % 4
//   x : chunk c (8 values) of row r at 16 r + (c ^ r)
// which spreads the 16 rows of an operand read over all banks.
template <int NB>
struct Stage {
    u32x4 w[NB][64];
    u32x4 x[256];
    uint32_t sc[NB * 16 * 8];   // scale dwords of 8 slices, [row][slice]
};

constexpr int kAhead = 4;       // slices of weights in flight

// A lane's addresses of the weights (row lane / 4 of each block) and scales.
template <int NB>
struct Weights {
    const uint8_t* w[NB];
    const uint8_t* s[2 * NB];
};

// Blocks at rows row0[b] .. + 16 of codes [.][K / 2] and scales [.][K / 32].
template <int NB>
__device__ __forceinline__ Weights<NB> weights_at(const uint8_t* w, const uint8_t* s, const size_t (&row0)[NB], int K) {
    const int lane = threadIdx.x & 63;
    Weights<NB> p;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        p.w[b] = w + (row0[b] + (lane >> 2)) * (size_t)(K / 2) + 16 * (((lane & 3) - (lane >> 4)) & 3);
#pragma unroll
        for (int i = 0; i < 2; ++i)   // entry lane + 64 i of the block's [16][8] scale dwords
            p.s[2 * b + i] = s + (row0[b] + 8 * i + (lane >> 3)) * (size_t)(K / 32);
    }
    return p;
}

// The first slices' weights and scales, [s0, s1), requested ahead of their use.
template <int NB>
struct Ahead {
    u32x4 w[kAhead][NB];
    uint32_t sc[2 * NB];
};

template <int NB>
__device__ __forceinline__ void load_scales(const Weights<NB>& p, int s, int s1, uint32_t (&sc)[2 * NB]) {
    const int sl = min(s + (int)(threadIdx.x & 7), s1 - 1);
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) sc[i] = *reinterpret_cast<const uint32_t*>(p.s[i] + 4 * sl);
}

template <int NB>
__device__ __forceinline__ void load_ahead(const Weights<NB>& p, int s0, int s1, Ahead<NB>& a) {
    if (s0 >= s1) return;
    load_scales<NB>(p, s0, s1, a.sc);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (s0 + u < s1) {
#pragma unroll
            for (int b = 0; b < NB; ++b) a.w[u][b] = *reinterpret_cast<const u32x4*>(p.w[b] + 64 * (s0 + u));
        }
}

// A lane's addresses of the activation rows: chunk lane % 16 of rows
// 4 j + lane / 16, j < nx.  Columns past the last row repeat it (or hold
// what the stage held): the columns of the product are independent, and theirs
// are not stored.
struct Acts {
    const uint16_t* x[4];
    int nx;
};

// acc[b] = the product over the 128-wide slices [s0, s1) of K, on top of acc.
template <int NB>
__device__ __forceinline__ void mma_slices(Stage<NB>& st, const Weights<NB>& p, Ahead<NB>& a, const Acts& in, int s0,
                                           int s1, f32x4 (&acc)[NB]) {
    const int lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
    u32x4 x[2][4];
    auto load_x = [&](int sl, u32x4 (&v)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < in.nx) v[j] = *reinterpret_cast<const u32x4*>(in.x[j] + 128 * sl);
    };
    if (s0 < s1) load_x(s0, x[0]);
    if (s0 + 1 < s1) load_x(s0 + 1, x[1]);
    for (int g = s0; g < s1; g += 8) {
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) st.sc[lane + 64 * i] = a.sc[i];
        if (g + 8 < s1) load_scales<NB>(p, g + 8, s1, a.sc);
        for (int h = g; h < min(g + 8, s1); h += kAhead) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int s = h + u;
                if (s >= s1) break;
#pragma unroll
                for (int b = 0; b < NB; ++b) st.w[b][lane] = a.w[u][b];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < in.nx) st.x[64 * j + 16 * q + (m ^ (4 * j + q))] = x[u & 1][j];
                if (s + kAhead < s1) {
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        a.w[u][b] = *reinterpret_cast<const u32x4*>(p.w[b] + 64 * (s + kAhead));
                }
                if (s + 2 < s1) load_x(s + 2, x[u & 1]);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                u32x4 wf[NB], xf[4];
                float sc[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    wf[b] = st.w[b][4 * m + ((q + (m >> 2)) & 3)];
                    sc[b] = e8m0_scale(reinterpret_cast<const uint8_t*>(st.sc)[((16 * b + m) * 8 + (s - g)) * 4 + q]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) xf[i] = st.x[16 * m + ((4 * q + i) ^ m)];
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp4_to_bf16(wf[b][i], sc[b]),
                                                                         __builtin_bit_cast(bf16x8, xf[i]), acc[b], 0,
                                                                         0, 0);
            }
        }
    }
}

// Rows rows[n0 .. n) of a list as a wave's activations: row r reads line
// r / div of x [.][K].
__device__ __forceinline__ Acts acts_at(const uint16_t* x, const uint16_t* rows, int n0, int n, int div, int K) {
    const int lane = threadIdx.x & 63;
    Acts in;
    in.nx = min(4, (n - n0 + 3) / 4);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        in.x[j] = x + (size_t)(rows[min(n0 + 4 * j + (lane >> 4), n - 1)] / div) * K + 8 * (lane & 15);
    return in;
}

// Two blocks of 16 weight rows (row0) times the group's rows, the waves of the
// workgroup taking the quarters of K: the quarters' sums of rows n0 .. + 16,
// added in order, to store(routed row, block 0, block 1) on wave 0's lanes.
template <typename Store>
__device__ __forceinline__ void group_product(GroupRows& s_g, Stage<2>* stage, const uint8_t* w, const uint8_t* s,
                                              const size_t (&row0)[2], const uint16_t* x, int n, int div, int K,
                                              Store store) {
    const int lane = threadIdx.x & 63, wave = wave_index(), m = lane & 15;
    const int ns = K / 128, sl0 = wave * ns / 4, sl1 = (wave + 1) * ns / 4;
    const Weights<2> p = weights_at<2>(w, s, row0, K);
    for (int n0 = 0; n0 < n; n0 += 16) {
        Ahead<2> a;
        load_ahead<2>(p, sl0, sl1, a);
        const Acts in = acts_at(x, s_g.rows, n0, n, div, K);
        f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        mma_slices<2>(stage[wave], p, a, in, sl0, sl1, acc);
        f32x4* red = reinterpret_cast<f32x4*>(stage[wave].x);
        red[lane] = acc[0];
        red[64 + lane] = acc[1];
        __syncthreads();
        if (wave == 0 && n0 + m < n) {
            f32x4 v[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                auto part = [&](int i) { return reinterpret_cast<const f32x4*>(stage[i].x)[64 * b + lane]; };
                v[b] = ((part(0) + part(1)) + part(2)) + part(3);
            }
            store((int)s_g.rows[n0 + m], v[0], v[1]);
        }
        if (n0 + 16 < n) __syncthreads();   // the stages are written again
    }
}

}  // namespace

// Gate and up projections: workgroup = (group, 16 hidden units);
// h[r] = silu(a) b as bfloat16.
__global__ __launch_bounds__(256) void decode_up_kernel(const uint16_t* __restrict__ x,
                                                        const int32_t* __restrict__ idx,
                                                        const uint8_t* __restrict__ w1,
                                                        const uint8_t* __restrict__ s1, uint16_t* __restrict__ h,
                                                        int R, int E, int k, int d, int H) {
    __shared__ GroupRows s_g;
    __shared__ Stage<2> stage[4];
    const int nb = H / 16, g = blockIdx.x / nb, hb = blockIdx.x - g * nb;
    int e;
    const int n = group_rows(idx, R, E, g, e, s_g);
    if (n == 0) return;
    // packed rows of hidden units 16 hb .. + 16: gate at 64 (hb / 2) + 16 (hb % 2), up 32 further
    const size_t row = (size_t)e * 2 * H + 64 * (hb >> 1) + 16 * (hb & 1);
    const int q = (threadIdx.x & 63) >> 4;
    group_product(s_g, stage, w1, s1, {row, row + 32}, x, n, k, d, [&](int r, const f32x4& a, const f32x4& b) {
        float o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = a[i] / (1.0f + expf(-a[i])) * b[i];
        *reinterpret_cast<uint2*>(h + (size_t)r * H + 16 * hb + 4 * q) =
            make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    });
}

// Down projection: workgroup = (group, 32 outputs), ye[r][d] in float32.
__global__ __launch_bounds__(256) void decode_down_kernel(const uint16_t* __restrict__ h,
                                                          const int32_t* __restrict__ idx,
                                                          const uint8_t* __restrict__ w2,
                                                          const uint8_t* __restrict__ s2, float* __restrict__ ye,
                                                          int R, int E, int d, int H) {
    __shared__ GroupRows s_g;
    __shared__ Stage<2> stage[4];
    const int nb = d / 32, g = blockIdx.x / nb, cb = blockIdx.x - g * nb;
    int e;
    const int n = group_rows(idx, R, E, g, e, s_g);
    if (n == 0) return;
    const size_t row = (size_t)e * d + 32 * cb;
    const int q = (threadIdx.x & 63) >> 4;
    group_product(s_g, stage, w2, s2, {row, row + 16}, h, n, 1, H, [&](int r, const f32x4& a, const f32x4& b) {
        float* dst = ye + (size_t)r * d + 32 * cb + 4 * q;
        *reinterpret_cast<f32x4*>(dst) = a;
        *reinterpret_cast<f32x4*>(dst + 16) = b;
    });
}

// y[t] = sum_j gate[t][j] ye[t k + j] in slot order over the slots in use
// (float32, rounded once); four outputs per thread.  Slots past k repeat slot
// k - 1, so that the loads need no branch and are in flight together.
template <int KMAX>
__global__ __launch_bounds__(256) void decode_combine_kernel(const float* __restrict__ ye,
                                                             const int32_t* __restrict__ idx,
                                                             const float* __restrict__ gate, uint16_t* __restrict__ y,
                                                             int E, int k, int d) {
    const int t = blockIdx.y, c = 4 * (blockIdx.x * 256 + threadIdx.x);
    if (c >= d) return;
    f32x4 v[KMAX];
    float g[KMAX];
    int e[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
        const int r = t * k + min(j, k - 1);
        e[j] = idx[r];
        g[j] = gate[r];
        v[j] = *reinterpret_cast<const f32x4*>(ye + (size_t)r * d + c);
    }
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
        if (j < k && e[j] >= 0 && e[j] < E) {   // ye of an unused slot was not written
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = fmaf(g[j], v[j][i], s[i]);
        }
    }
    *reinterpret_cast<uint2*>(y + (size_t)t * d + c) = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
}

// Down projection and combine of few rows: workgroup = (token, 16 outputs),
// sixteen waves, a wave per quarter of a slot in turn (the slot's h the only
// column).  No float32 rows and no third launch, but tokens that share an
// expert each read its weights.
__global__ __launch_bounds__(1024) void decode_down_token_kernel(const uint16_t* __restrict__ h,
                                                                 const int32_t* __restrict__ idx,
                                                                 const float* __restrict__ gate,
                                                                 const uint8_t* __restrict__ w2,
                                                                 const uint8_t* __restrict__ s2,
                                                                 uint16_t* __restrict__ y, int E, int k, int d, int H) {
    __shared__ Stage<1> stage[16];
    __shared__ float red[kMaxTopK][4][16];
    __shared__ float s_gate[kMaxTopK];
    const int lane = threadIdx.x & 63, wave = wave_index(), m = lane & 15, q = lane >> 4;
    const int nb = d / 16, t = blockIdx.x / nb, cb = blockIdx.x - t * nb;
    const int ns = H / 128;
    for (int u = wave; u < 4 * k; u += 16) {
        const int j = u >> 2, quarter = u & 3, r = t * k + j, e = uniform(idx[r]);
        const bool used = e >= 0 && e < E;
        f32x4 acc[1] = {{0.f, 0.f, 0.f, 0.f}};
        if (used) {
            const int sl0 = quarter * ns / 4, sl1 = (quarter + 1) * ns / 4;
            const Weights<1> p = weights_at<1>(w2, s2, {(size_t)e * d + 16 * cb}, H);
            Ahead<1> a;
            load_ahead<1>(p, sl0, sl1, a);
            const uint16_t* hr = h + (size_t)r * H + 8 * m;
            mma_slices<1>(stage[wave], p, a, {{hr, hr, hr, hr}, 1}, sl0, sl1, acc);
        }
        if (m == 0) *reinterpret_cast<f32x4*>(&red[j][quarter][4 * q]) = acc[0];
        if (lane == 0 && quarter == 0) s_gate[j] = used ? gate[r] : 0.f;
    }
    __syncthreads();
    if (threadIdx.x < 16) {
        const int c = threadIdx.x;
        float s = 0.f;
        for (int j = 0; j < k; ++j)
            s = fmaf(s_gate[j], ((red[j][0][c] + red[j][1][c]) + red[j][2][c]) + red[j][3][c], s);
        y[(size_t)t * d + 16 * cb + c] = f32_to_bf16(s);
    }
}

// E2M1 code of v: round to nearest even, saturate to +-6, keep the sign on zero.
__device__ __forceinline__ uint32_t e2m1_encode(float v) {
    const uint32_t sign = (__float_as_uint(v) >> 28) & 8u;
    const float a = fminf(fabsf(v), 6.0f);
    // steps 1/2 below 2, 1 below 4, 2 to 6: rintf rounds halves to even, and
    // an even multiple of the step is an even code
    const float c = a < 2.0f ? rintf(a * 2.0f) : (a < 4.0f ? rintf(a) + 2.0f : rintf(a * 0.5f) + 4.0f);
    return sign | (uint32_t)c;
}

// MXFP4 of bfloat16 weights [E][K][N] (the x . W convention): destination row
// n holds column n, a thread one scale block of 32 k of it.  Shared exponent
// floor(log2(amax)) - 2, clamped to [-127, 127].  GU: the destination rows are
// W1's, gathered from gate (a) and up (b).  Setup, not timed.
template <bool GU>
__global__ __launch_bounds__(256) void pack_mxfp4_kernel(const uint16_t* __restrict__ a,
                                                         const uint16_t* __restrict__ b, int E, int K, int N,
                                                         uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    const int rows = GU ? 2 * N : N;
    const int nb = (rows + 255) / 256, kb = blockIdx.x / nb, e = blockIdx.y;
    const int n = (int)(blockIdx.x - kb * nb) * 256 + threadIdx.x;
    if (n >= rows) return;
    // destination row n of W1: gate column h = 32 (n / 64) + n % 32 when (n / 32) is even, else up column h
    const int col = GU ? 32 * (n >> 6) + (n & 31) : n;
    const uint16_t* src = (GU && ((n >> 5) & 1) ? b : a) + ((size_t)e * K + 32 * kb) * N + col;
    float v[32], amax = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        v[i] = bf16_to_f32(src[(size_t)i * N]);
        amax = fmaxf(amax, fabsf(v[i]));
    }
    const int ef = (int)((__float_as_uint(amax) >> 23) & 0xFF);
    const int se = ef == 0 ? -127 : max(ef - 127 - 2, -127);
    // v 2^-se in two exact steps: 2^127 is the largest float32 power
    const float s0 = __uint_as_float((uint32_t)(127 - se / 2) << 23), s1 = __uint_as_float((uint32_t)(127 - (se - se / 2)) << 23);
    u32x4 o = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i / 8] |= e2m1_encode(v[i] * s0 * s1) << (4 * (i % 8));
    const size_t row = (size_t)e * rows + n;
    *reinterpret_cast<u32x4*>(codes + row * (K / 2) + 16 * kb) = o;
    scales[row * (K / 32) + kb] = (uint8_t)(se + 127);
}

hipError_t launch_pack_mxfp4(const void* w_gate, const void* w_up, const void* w_down, uint8_t* w1, uint8_t* w2,
                             uint8_t* s1, uint8_t* s2, int E, int d, int H, hipStream_t s) {
    hipLaunchKernelGGL((pack_mxfp4_kernel<true>), dim3((2 * H + 255) / 256 * (d / 32), E), dim3(256), 0, s,
                       static_cast<const uint16_t*>(w_gate), static_cast<const uint16_t*>(w_up), E, d, H, w1, s1);
    hipLaunchKernelGGL((pack_mxfp4_kernel<false>), dim3((d + 255) / 256 * (H / 32), E), dim3(256), 0, s,
                       static_cast<const uint16_t*>(w_down), nullptr, E, H, d, w2, s2);
    return hipGetLastError();
}

hipError_t launch_decode_experts(const uint16_t* x, const int32_t* idx, const float* gate, const uint8_t* w1,
                                 const uint8_t* w2, const uint8_t* s1, const uint8_t* s2, uint16_t* h, float* ye,
                                 uint16_t* y, int T, int d, int E, int k, int H, hipStream_t s) {
    const int R = T * k, G = R <= E ? R : E;
    hipLaunchKernelGGL(decode_up_kernel, dim3(G * (H / 16)), dim3(256), 0, s, x, idx, w1, s1, h, R, E, k, d, H);
    if (2 * R <= E) {
        hipLaunchKernelGGL(decode_down_token_kernel, dim3(T * (d / 16)), dim3(1024), 0, s, h, idx, gate, w2, s2, y, E, k,
                           d, H);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(decode_down_kernel, dim3(G * (d / 32)), dim3(256), 0, s, h, idx, w2, s2, ye, R, E, d, H);
    const dim3 cg((d / 4 + 255) / 256, T), cb(256);
    if (k <= 4) hipLaunchKernelGGL(decode_combine_kernel<4>, cg, cb, 0, s, ye, idx, gate, y, E, k, d);
    else if (k <= 8) hipLaunchKernelGGL(decode_combine_kernel<8>, cg, cb, 0, s, ye, idx, gate, y, E, k, d);
    else hipLaunchKernelGGL(decode_combine_kernel<kMaxTopK>, cg, cb, 0, s, ye, idx, gate, y, E, k, d);
    return hipGetLastError();
}

}  // namespace moe
