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
// x stays bfloat16.  h goes through memory as two bfloat16 terms (the rounded
// value and the rounded remainder, 2^-16 of it left out): rounded once it would
// add as much error to y as y's own rounding, and the second term costs loads
// that hit the caches and matrix instructions that the weights' bytes hide.
// Rows are not sorted or moved: a workgroup finds its expert's rows in topk_idx
// itself, and an index outside [0, E) is a slot not in use.
//
// Every sum over K is taken in four quarters (of K / 128 slices, in order) that
// are added in order, whichever kernel and however many rows: a token's result
// does not depend on the tokens beside it.
//
// The weights' bytes bound it.  d = 4096, E = 64, k = 8, H = 1536: one token 20 us
// (80 MB, 3.9 TB/s), 64 tokens 144 us (643 MB, 4.5 TB/s); T = 7, d = 2048, E = 128,
// k = 4, H = 1024: 20 us (63 MB, 3.1 TB/s; two launches of 2.5 us and more whatever
// they read).  A 2 GiB copy runs at 4.9 TB/s on the same card.
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
    int32_t cnt[4][4];
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
    for (int base = 0; base < R; base += 1024) {   // 1024 rows at a time: their loads together, two barriers
        int v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = idx[min(base + 256 * i + tid, R - 1)];
        uint64_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b[i] = __ballot(v[i] == expert && base + 256 * i + tid < R);
            if (lane == 0) s.cnt[i][wave] = __popcll(b[i]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int off = n, all = n;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int c = s.cnt[i][w];
                if (w < wave) off += c;
                all += c;
            }
            if (b[i] >> lane & 1) s.rows[off + __popcll(b[i] & ((1ull << lane) - 1ull))] = (uint16_t)(base + 256 * i + tid);
            n = uniform(all);
        }
        __syncthreads();   // cnt is rewritten by the next rows; rows[] is complete after the last
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
// XR rows of activations are staged (1, 4 or 16), each of NT terms (row r of
// term n at XR n + r); column m of the product reads row m % XR.
template <int NB, int XR, int NT>
struct Stage {
    u32x4 w[NB][64];
    u32x4 x[16 * XR * NT];
    uint32_t sc[NB * 16 * 8];   // scale dwords of 8 slices, [row][slice]
};

// 16 bytes or a dword at a uniform address plus a lane's 32-bit offset (an
// expert's weights and an activation buffer are below 2^32 bytes).
__device__ __forceinline__ u32x4 load16(const uint8_t* base, uint32_t off) {
    return *reinterpret_cast<const u32x4*>(base + off);
}
__device__ __forceinline__ uint32_t load4(const uint8_t* base, uint32_t off) {
    return *reinterpret_cast<const uint32_t*>(base + off);
}

// Weight rows row0[b] .. + 16 of an expert's codes w [.][K / 2] and scales
// s [.][K / 32], and a lane's offsets: row lane / 4 of each block's codes,
// entries lane and lane + 64 of its [16][8] scale dwords (rows lane / 8 and
// 8 further).
template <int NB>
struct Weights {
    const uint8_t* w[NB];
    const uint8_t* s[2 * NB];
    uint32_t wo, so;
};

template <int NB>
__device__ __forceinline__ Weights<NB> weights_at(const uint8_t* w, const uint8_t* s, const int (&row0)[NB], int K) {
    const int lane = threadIdx.x & 63;
    Weights<NB> p;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        p.w[b] = w + (size_t)row0[b] * (K / 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) p.s[2 * b + i] = s + (size_t)(row0[b] + 8 * i) * (K / 32);
    }
    p.wo = (uint32_t)(lane >> 2) * (uint32_t)(K / 2) + 16 * (((lane & 3) - (lane >> 4)) & 3);
    p.so = (uint32_t)(lane >> 3) * (uint32_t)(K / 32);
    return p;
}

// Loads of an activation slice: four staged rows each.
constexpr int x_loads(int XR, int NT) { return (XR * NT + 3) / 4; }

// Requests in flight: D slices of weights and of activations (loads return in
// order, so a slice of one kind waits for those of the other requested before
// it: both have the same depth), and the next 8 slices' scales.
template <int NB, int XR, int NT, int D>
struct Ahead {
    u32x4 w[D][NB], x[D][x_loads(XR, NT)];
    uint32_t sc[2 * NB];
};

template <int NB>
__device__ __forceinline__ void load_scales(const Weights<NB>& p, int s, int s1, uint32_t (&sc)[2 * NB]) {
    const int sl = min(s + (int)(threadIdx.x & 7), s1 - 1);
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) sc[i] = load4(p.s[i], p.so + 4 * sl);
}

// Activation rows: a lane's offsets of chunk lane % 16 of staged rows
// 4 j + lane / 16.  Of a term's loads the first nx have a row to bring (XR < 16:
// all).  Columns past the last row repeat it (or hold what the stage held): the
// columns of the product are independent, and theirs are not stored.
template <int XR, int NT>
struct Acts {
    const uint8_t* x;
    uint32_t xo[x_loads(XR, NT)];
    int nx;
};

template <int XR>
__device__ __forceinline__ bool brings(int j, int nx) {
    return XR < 16 || j % (XR / 4) < nx;
}

template <int NB, int XR, int NT>
__device__ __forceinline__ void load_slice(const Weights<NB>& p, const Acts<XR, NT>& in, int s, u32x4 (&w)[NB],
                                           u32x4 (&x)[x_loads(XR, NT)]) {
#pragma unroll
    for (int b = 0; b < NB; ++b) w[b] = load16(p.w[b] + 64 * s, p.wo);
#pragma unroll
    for (int j = 0; j < x_loads(XR, NT); ++j)
        if (brings<XR>(j, in.nx)) x[j] = load16(in.x + 256 * s, in.xo[j]);
}

template <int NB, int XR, int NT, int D>
__device__ __forceinline__ void load_ahead(const Weights<NB>& p, const Acts<XR, NT>& in, int s0, int s1,
                                           Ahead<NB, XR, NT, D>& a) {
    if (s0 >= s1) return;
    load_scales<NB>(p, s0, s1, a.sc);
#pragma unroll
    for (int u = 0; u < D; ++u)
        if (s0 + u < s1) load_slice<NB, XR, NT>(p, in, s0 + u, a.w[u], a.x[u]);
}

// acc[b] = the product over the 128-wide slices [s0, s1) of K, on top of acc.
template <int NB, int XR, int NT, int D>
__device__ __forceinline__ void mma_slices(Stage<NB, XR, NT>& st, const Weights<NB>& p, Ahead<NB, XR, NT, D>& a,
                                           const Acts<XR, NT>& in, int s0, int s1, f32x4 (&acc)[NB]) {
    static_assert(8 % D == 0, "a group of 8 slices' scales is whole rounds of requests");
    const int lane = threadIdx.x & 63, m = lane & 15, q = lane >> 4;
    for (int g = s0; g < s1; g += 8) {
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) st.sc[lane + 64 * i] = a.sc[i];
        if (g + 8 < s1) load_scales<NB>(p, g + 8, s1, a.sc);
        for (int h = g; h < min(g + 8, s1); h += D) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
                const int s = h + u;
                if (s >= s1) break;
#pragma unroll
                for (int b = 0; b < NB; ++b) st.w[b][lane] = a.w[u][b];
#pragma unroll
                for (int j = 0; j < x_loads(XR, NT); ++j) {
                    // fewer than four staged rows: lanes of the same row store the same
                    const int r = (4 * j + q) % (XR * NT);
                    if (brings<XR>(j, in.nx)) st.x[16 * r + (m ^ (r % XR))] = a.x[u][j];
                }
                if (s + D < s1) load_slice<NB, XR, NT>(p, in, s + D, a.w[u], a.x[u]);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                u32x4 wf[NB], xf[NT][4];
                float sc[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    wf[b] = st.w[b][4 * m + ((q + (m >> 2)) & 3)];
                    sc[b] = e8m0_scale(reinterpret_cast<const uint8_t*>(st.sc)[((16 * b + m) * 8 + (s - g)) * 4 + q]);
                }
                const int r = m & (XR - 1);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) xf[n][i] = st.x[16 * (XR * n + r) + ((4 * q + i) ^ r)];
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const bf16x8 wv = fp4_to_bf16(wf[b][i], sc[b]);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, __builtin_bit_cast(bf16x8, xf[n][i]),
                                                                             acc[b], 0, 0, 0);
                    }
            }
        }
    }
}

// Rows rows[n0 .. n) of a list as a wave's activations: row r reads line
// r / div of x [.][NT][K].
template <int XR, int NT>
__device__ __forceinline__ Acts<XR, NT> acts_at(const uint16_t* x, const uint16_t* rows, int n0, int n, int div,
                                                int K) {
    const int lane = threadIdx.x & 63;
    Acts<XR, NT> in;
    in.x = reinterpret_cast<const uint8_t*>(x);
    in.nx = min(XR / 4, (n - n0 + 3) / 4);
#pragma unroll
    for (int j = 0; j < XR / 4; ++j) {
        const uint32_t line = (uint32_t)(rows[min(n0 + 4 * j + (lane >> 4), n - 1)] / div);
#pragma unroll
        for (int t = 0; t < NT; ++t)
            in.xo[t * (XR / 4) + j] = (line * NT + t) * (uint32_t)(2 * K) + 16 * (lane & 15);
    }
    return in;
}

// NB blocks of 16 of the expert's weight rows (p) times the group's rows, XR at
// a time, the waves of the workgroup taking the quarters of K.  Each wave then
// calls store(routed row, sum), sum(b) being block b's product with this lane's
// column (the quarters added in order), on the columns that hold a row.  The
// next rows' first loads are in flight while a product is reduced and stored.
template <int NB, int XR, int NT, int D, typename Store>
__device__ __forceinline__ void group_product(GroupRows& s_g, Stage<NB, XR, NT>* stage, const Weights<NB>& p,
                                              const uint16_t* x, int n, int div, int K, Store store) {
    const int lane = threadIdx.x & 63, wave = wave_index(), m = lane & 15;
    const int ns = K / 128, sl0 = wave * ns / 4, sl1 = (wave + 1) * ns / 4;
    Acts<XR, NT> in = acts_at<XR, NT>(x, s_g.rows, 0, n, div, K);
    Ahead<NB, XR, NT, D> a;
    load_ahead<NB, XR, NT, D>(p, in, sl0, sl1, a);
    for (int n0 = 0; n0 < n; n0 += XR) {
        f32x4 acc[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
        mma_slices<NB, XR, NT, D>(stage[wave], p, a, in, sl0, sl1, acc);
        const bool more = n0 + XR < n;
        if (more) {
            in = acts_at<XR, NT>(x, s_g.rows, n0 + XR, n, div, K);
            load_ahead<NB, XR, NT, D>(p, in, sl0, sl1, a);
        }
        f32x4* red = reinterpret_cast<f32x4*>(stage[wave].w);
#pragma unroll
        for (int b = 0; b < NB; ++b) red[64 * b + lane] = acc[b];
        __syncthreads();
        if (m < XR && n0 + m < n) {
            store((int)s_g.rows[n0 + m], [&](int b) {
                auto part = [&](int i) { return reinterpret_cast<const f32x4*>(stage[i].w)[64 * b + lane]; };
                return ((part(0) + part(1)) + part(2)) + part(3);
            });
        }
        if (more) __syncthreads();   // the stages are written again
    }
}

// The same product with the waves side by side: each takes 16 NB weight rows of
// its own (p) and all of K, and the activations, up to 32 routed rows at a time,
// pass through LDS once for the four of them, two buffers deep with a barrier a
// slice.  With many rows an expert the activations' loads (two terms of h: as
// many bytes as the weights) held the memory pipe more than the weights':
// without them the quarters' kernels took 138 us instead of 164 (T = 64,
// d = 4096, E = 64, k = 8, H = 1536).  More than 16 rows take their weights'
// one reading together.
template <int NB, int NT>
struct WideStage {
    u32x4 x[2][2 * 16 * 16 * NT];
    u32x4 w[4][NB][64];
    uint32_t sc[4][NB * 16 * 8];
};

// RB blocks of 16 routed rows; calls store(routed row, the NB blocks' sums) on
// the columns that hold a row.
template <int NB, int NT, int RB, int D, typename Store>
__device__ __forceinline__ void wide_product(GroupRows& s_g, WideStage<NB, NT>& st, const Weights<NB>& p,
                                             const uint16_t* x, int n, int div, int K, Store store) {
    static_assert(D % 2 == 0, "a slice's buffer is its place in a round of requests");
    const int lane = threadIdx.x & 63, wave = wave_index(), m = lane & 15, q = lane >> 4;
    const int ns = K / 128, xr = 4 * wave + q;   // the row of each block that this lane brings
    for (int n0 = 0; n0 < n; n0 += 16 * RB) {
        uint32_t xo[RB];
        bool brings[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            brings[r] = 16 * r + 4 * wave < n - n0;
            xo[r] = (uint32_t)(s_g.rows[min(n0 + 16 * r + xr, n - 1)] / div) * (uint32_t)(2 * K * NT) + 16 * m;
        }
        u32x4 wr[D][NB], ar[D][RB][NT];
        uint32_t scr[2 * NB];
        auto load = [&](int sl, u32x4 (&wr)[NB], u32x4 (&ar)[RB][NT]) {
#pragma unroll
            for (int b = 0; b < NB; ++b) wr[b] = load16(p.w[b] + 64 * sl, p.wo);
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                if (!brings[r]) continue;
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    ar[r][t] = load16(reinterpret_cast<const uint8_t*>(x) + 2 * K * t + 256 * sl, xo[r]);
            }
        };
        load_scales<NB>(p, 0, ns, scr);
#pragma unroll
        for (int u = 0; u < D; ++u)
            if (u < ns) load(u, wr[u], ar[u]);
        f32x4 acc[RB][NB], sum[RB][NB];
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[r][b] = sum[r][b] = (f32x4){0.f, 0.f, 0.f, 0.f};
        int quarter = 1;   // the quarter that the next slice is in
        while (quarter * ns / 4 == 0) ++quarter;
        for (int g = 0; g < ns; g += 8) {
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) st.sc[wave][lane + 64 * i] = scr[i];
            if (g + 8 < ns) load_scales<NB>(p, g + 8, ns, scr);
            for (int h = g; h < min(g + 8, ns); h += D) {
#pragma unroll
                for (int u = 0; u < D; ++u) {
                    const int sl = h + u;
                    if (sl >= ns) break;
#pragma unroll
                    for (int b = 0; b < NB; ++b) st.w[wave][b][lane] = wr[u][b];
#pragma unroll
                    for (int r = 0; r < RB; ++r) {
                        if (!brings[r]) continue;
#pragma unroll
                        for (int t = 0; t < NT; ++t) st.x[u & 1][16 * (16 * (r * NT + t) + xr) + (m ^ xr)] = ar[u][r][t];
                    }
                    if (sl + D < ns) load(sl + D, wr[u], ar[u]);
                    __syncthreads();   // also: every wave has left the buffer that is written next
                    u32x4 wf[NB];
                    float sc[NB];
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        wf[b] = st.w[wave][b][4 * m + ((q + (m >> 2)) & 3)];
                        sc[b] = e8m0_scale(
                            reinterpret_cast<const uint8_t*>(st.sc[wave])[((16 * b + m) * 8 + (sl - g)) * 4 + q]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        bf16x8 xf[RB][NT];
#pragma unroll
                        for (int r = 0; r < RB; ++r)
#pragma unroll
                            for (int t = 0; t < NT; ++t)
                                xf[r][t] = __builtin_bit_cast(
                                    bf16x8, st.x[u & 1][16 * (16 * (r * NT + t) + m) + ((4 * q + i) ^ m)]);
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const bf16x8 wv = fp4_to_bf16(wf[b][i], sc[b]);
#pragma unroll
                            for (int r = 0; r < RB; ++r)
#pragma unroll
                                for (int t = 0; t < NT; ++t)
                                    acc[r][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, xf[r][t], acc[r][b], 0, 0, 0);
                        }
                    }
                    if (sl + 1 == quarter * ns / 4) {   // the quarters' sums, added in order
#pragma unroll
                        for (int r = 0; r < RB; ++r)
#pragma unroll
                            for (int b = 0; b < NB; ++b) {
                                sum[r][b] += acc[r][b];
                                acc[r][b] = (f32x4){0.f, 0.f, 0.f, 0.f};
                            }
                    }
                    while (quarter < 4 && sl + 1 >= quarter * ns / 4) ++quarter;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < RB; ++r)
            if (n0 + 16 * r + m < n) store((int)s_g.rows[n0 + 16 * r + m], sum[r]);
        if (n0 + 16 * RB < n) __syncthreads();   // the buffers are written again
    }
}

// silu(a) b of four hidden units as two bfloat16 terms, at dst and H further.
// The first term ends at bfloat16's largest value: rounded on to infinity, the
// remainder would be -inf and the products' sum NaN.  (An infinite or NaN value
// is its second term.)  The remainder is that of the rounded product in every
// kernel: without the pragma one of them may fuse the two operations.
__device__ __forceinline__ void store_h(const f32x4& a, const f32x4& b, uint16_t* dst, int H) {
#pragma clang fp contract(off)
    constexpr float kMax = 0x1.fep127f;
    float hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float o = a[i] / (1.0f + expf(-a[i])) * b[i];
        hi[i] = bf16_round(fminf(fmaxf(o, -kMax), kMax));
        lo[i] = o - hi[i];
    }
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3]));
    *reinterpret_cast<uint2*>(dst + H) = make_uint2(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]));
}

}  // namespace

// Gate and up projections: workgroup = (group, 8 NB hidden units), half of its
// weight rows the gate's, half the up's; h[r] = silu(a) b as two terms.
template <int NB, int XR, int D>
__global__ __launch_bounds__(256) void decode_up_kernel(const uint16_t* __restrict__ x,
                                                        const int32_t* __restrict__ idx,
                                                        const uint8_t* __restrict__ w1,
                                                        const uint8_t* __restrict__ s1, uint16_t* __restrict__ h,
                                                        int R, int E, int k, int d, int H) {
    __shared__ GroupRows s_g;
    __shared__ Stage<NB, XR, 1> stage[4];
    const int nb = H / (8 * NB), g = blockIdx.x / nb, hb = blockIdx.x - g * nb;
    int e;
    const int n = group_rows(idx, R, E, g, e, s_g);
    if (n == 0) return;
    // packed rows of hidden unit u: gate at 64 (u / 32) + u % 32, up 32 further
    const int u0 = 8 * NB * hb, wave = wave_index(), q = (threadIdx.x & 63) >> 4;
    int row0[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) row0[b] = 64 * (u0 / 32) + u0 % 32 + 16 * (b % (NB / 2)) + 32 * (b / (NB / 2));
    const Weights<NB> p = weights_at<NB>(w1 + (size_t)e * H * d, s1 + (size_t)e * H * (d / 16), row0, d);
    group_product<NB, XR, 1, D>(s_g, stage, p, x, n, k, d, [&](int r, auto sum) {
        if (wave >= NB / 2) return;   // wave b: hidden units u0 + 16 b .. + 16
        store_h(sum(wave), sum(wave + NB / 2), h + (size_t)r * 2 * H + u0 + 16 * wave + 4 * q, H);
    });
}

// Down projection: workgroup = (group, 16 NB outputs), ye[r][d] in float32.
template <int NB, int XR, int D>
__global__ __launch_bounds__(256) void decode_down_kernel(const uint16_t* __restrict__ h,
                                                          const int32_t* __restrict__ idx,
                                                          const uint8_t* __restrict__ w2,
                                                          const uint8_t* __restrict__ s2, float* __restrict__ ye,
                                                          int R, int E, int d, int H) {
    __shared__ GroupRows s_g;
    __shared__ Stage<NB, XR, 2> stage[4];
    const int nb = d / (16 * NB), g = blockIdx.x / nb, cb = blockIdx.x - g * nb;
    int e;
    const int n = group_rows(idx, R, E, g, e, s_g);
    if (n == 0) return;
    const int c0 = 16 * NB * cb, wave = wave_index(), q = (threadIdx.x & 63) >> 4;
    int row0[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) row0[b] = c0 + 16 * b;
    const Weights<NB> p = weights_at<NB>(w2 + (size_t)e * d * (H / 2), s2 + (size_t)e * d * (H / 32), row0, H);
    group_product<NB, XR, 2, D>(s_g, stage, p, h, n, 1, H, [&](int r, auto sum) {
        if (wave < NB) *reinterpret_cast<f32x4*>(ye + (size_t)r * d + c0 + 16 * wave + 4 * q) = sum(wave);
    });
}

// The two projections with the waves side by side: 32 NB hidden units, 64 NB outputs a workgroup.
template <int NB, int D>
__global__ __launch_bounds__(256, 3) void decode_up_wide_kernel(const uint16_t* __restrict__ x,
                                                                const int32_t* __restrict__ idx,
                                                                const uint8_t* __restrict__ w1,
                                                                const uint8_t* __restrict__ s1,
                                                                uint16_t* __restrict__ h, int R, int E, int k, int d,
                                                                int H) {
    __shared__ GroupRows s_g;
    __shared__ WideStage<NB, 1> stage;
    const int nb = H / (32 * NB), g = blockIdx.x / nb, hb = blockIdx.x - g * nb;
    int e;
    const int n = group_rows(idx, R, E, g, e, s_g);
    if (n == 0) return;
    const int u0 = 32 * NB * hb + 8 * NB * wave_index(), q = (threadIdx.x & 63) >> 4;
    int row0[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) row0[b] = 64 * (u0 / 32) + u0 % 32 + 16 * (b % (NB / 2)) + 32 * (b / (NB / 2));
    const Weights<NB> p = weights_at<NB>(w1 + (size_t)e * H * d, s1 + (size_t)e * H * (d / 16), row0, d);
    auto store = [&](int r, const f32x4 (&sum)[NB]) {
#pragma unroll
        for (int b = 0; b < NB / 2; ++b) store_h(sum[b], sum[b + NB / 2], h + (size_t)r * 2 * H + u0 + 16 * b + 4 * q, H);
    };
    if (n > 16) wide_product<NB, 1, 2, D>(s_g, stage, p, x, n, k, d, store);
    else wide_product<NB, 1, 1, D>(s_g, stage, p, x, n, k, d, store);
}

template <int NB, int D>
__global__ __launch_bounds__(256, 3) void decode_down_wide_kernel(const uint16_t* __restrict__ h,
                                                                  const int32_t* __restrict__ idx,
                                                                  const uint8_t* __restrict__ w2,
                                                                  const uint8_t* __restrict__ s2,
                                                                  float* __restrict__ ye, int R, int E, int d, int H) {
    __shared__ GroupRows s_g;
    __shared__ WideStage<NB, 2> stage;
    const int nb = d / (64 * NB), g = blockIdx.x / nb, cb = blockIdx.x - g * nb;
    int e;
    const int n = group_rows(idx, R, E, g, e, s_g);
    if (n == 0) return;
    const int c0 = 64 * NB * cb + 16 * NB * wave_index(), q = (threadIdx.x & 63) >> 4;
    int row0[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) row0[b] = c0 + 16 * b;
    const Weights<NB> p = weights_at<NB>(w2 + (size_t)e * d * (H / 2), s2 + (size_t)e * d * (H / 32), row0, H);
    auto store = [&](int r, const f32x4 (&sum)[NB]) {
#pragma unroll
        for (int b = 0; b < NB; ++b) *reinterpret_cast<f32x4*>(ye + (size_t)r * d + c0 + 16 * b + 4 * q) = sum[b];
    };
    if (n > 16) wide_product<NB, 2, 2, D>(s_g, stage, p, h, n, 1, H, store);
    else wide_product<NB, 2, 1, D>(s_g, stage, p, h, n, 1, H, store);
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

// Down projection and combine of few rows: workgroup = (token, 16 NB outputs),
// sixteen waves, a wave per quarter of a slot in turn (the slot's h in every
// column).  No float32 rows and no third launch, but tokens that share an
// expert each read its weights.
template <int NB, int D>
__global__ __launch_bounds__(1024) void decode_down_token_kernel(const uint16_t* __restrict__ h,
                                                                 const int32_t* __restrict__ idx,
                                                                 const float* __restrict__ gate,
                                                                 const uint8_t* __restrict__ w2,
                                                                 const uint8_t* __restrict__ s2,
                                                                 uint16_t* __restrict__ y, int E, int k, int d, int H) {
    __shared__ Stage<NB, 1, 2> stage[16];
    __shared__ float red[kMaxTopK][4][16 * NB];
    __shared__ float s_gate[kMaxTopK];
    const int lane = threadIdx.x & 63, wave = wave_index(), m = lane & 15, q = lane >> 4;
    const int nb = d / (16 * NB), t = blockIdx.x / nb, cb = blockIdx.x - t * nb;
    const int ns = H / 128, quarter = wave & 3, sl0 = quarter * ns / 4, sl1 = (quarter + 1) * ns / 4;
    int row0[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) row0[b] = 16 * (NB * cb + b);
    // slot j of this wave: its expert's weights and h requested, -1 if it is not in use
    auto request = [&](int j, Weights<NB>& p, Acts<1, 2>& in, Ahead<NB, 1, 2, D>& a) {
        const int e = uniform(idx[t * k + j]);
        if (e < 0 || e >= E) return -1;
        p = weights_at<NB>(w2 + (size_t)e * d * (H / 2), s2 + (size_t)e * d * (H / 32), row0, H);
        in = {reinterpret_cast<const uint8_t*>(h), {(uint32_t)(2 * (t * k + j) + (q & 1)) * (uint32_t)(2 * H) + 16 * m}, 1};
        load_ahead<NB, 1, 2, D>(p, in, sl0, sl1, a);
        return e;
    };
    Weights<NB> p;
    Acts<1, 2> in;
    Ahead<NB, 1, 2, D> a;
    for (int j = wave >> 2; j < k; j += 4) {
        const int e = request(j, p, in, a);
        f32x4 acc[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
        if (e >= 0) mma_slices<NB, 1, 2, D>(stage[wave], p, a, in, sl0, sl1, acc);
        if (m == 0) {
#pragma unroll
            for (int b = 0; b < NB; ++b) *reinterpret_cast<f32x4*>(&red[j][quarter][16 * b + 4 * q]) = acc[b];
        }
        if (lane == 0 && quarter == 0) s_gate[j] = e >= 0 ? gate[t * k + j] : 0.f;
    }
    __syncthreads();
    if (threadIdx.x < 16 * NB) {
        const int c = threadIdx.x;
        float s = 0.f;
        for (int j = 0; j < k; ++j)
            s = fmaf(s_gate[j], ((red[j][0][c] + red[j][1][c]) + red[j][2][c]) + red[j][3][c], s);
        y[(size_t)t * d + 16 * NB * cb + c] = f32_to_bf16(s);
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
// floor(log2(amax)) - 2, clamped to [-127, 127]; 255, the scale that is NaN, for a
// block with a NaN.  GU: the destination rows are W1's, gathered from gate (a)
// and up (b).  Setup, not timed.
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
    bool nan = false;   // fmaxf passes it over, and E2M1 has no code for it
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        v[i] = bf16_to_f32(src[(size_t)i * N]);
        amax = fmaxf(amax, fabsf(v[i]));
        nan |= v[i] != v[i];
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
    scales[row * (K / 32) + kb] = nan ? (uint8_t)255 : (uint8_t)(se + 127);
}

hipError_t launch_pack_mxfp4(const void* w_gate, const void* w_up, const void* w_down, uint8_t* w1, uint8_t* w2,
                             uint8_t* s1, uint8_t* s2, int E, int d, int H, hipStream_t s) {
    hipLaunchKernelGGL((pack_mxfp4_kernel<true>), dim3((2 * H + 255) / 256 * (d / 32), E), dim3(256), 0, s,
                       static_cast<const uint16_t*>(w_gate), static_cast<const uint16_t*>(w_up), E, d, H, w1, s1);
    hipLaunchKernelGGL((pack_mxfp4_kernel<false>), dim3((d + 255) / 256 * (H / 32), E), dim3(256), 0, s,
                       static_cast<const uint16_t*>(w_down), nullptr, E, H, d, w2, s2);
    return hipGetLastError();
}

// Workgroups from which the kernels with their waves side by side are taken:
// two on every compute unit.  T = 64, d = 4096, E = 64, k = 8, H = 1536 (1536
// and 2048 of them): the kernels together 151 us against 171 with the waves on
// the quarters of K, T = 256: 302 and 372; T = 16, E = 8, k = 2, H = 1536 (192
// and 256): 18.4 + 10.5 us the two products against 13.2 + 9.3.
// With no more rows than experts a group mostly holds one row, few activations
// to share: the up projection then keeps its waves on the quarters (T = 12,
// d = 4096, E = 64, k = 4, H = 1536: 46 us against 55); the down projection, with
// two terms of h and a short K, does not (34 against 31).
// Up to half as many rows as experts a token's workgroup joins its own slots,
// which saves ye and a launch and reads shared experts again: T = 1, k = 8: 8.3
// us against 9.0 + 3.9, T = 4: 27 against 25 + 5, T = 6 (48 rows): 41 against
// 31 + 5.  It takes 16 outputs rather than 32 where 32 give fewer workgroups
// than compute units: T = 1: 8.3 us against 11.6, T = 2: 16.0 against 14.1.
constexpr int kWideGroups = 512;

hipError_t launch_decode_experts(const uint16_t* x, const int32_t* idx, const float* gate, const uint8_t* w1,
                                 const uint8_t* w2, const uint8_t* s1, const uint8_t* s2, uint16_t* h, float* ye,
                                 uint16_t* y, int T, int d, int E, int k, int H, hipStream_t s) {
    const int R = T * k, G = R <= E ? R : E;
    const dim3 wg(256);
    const int up = G * (H / 64), down = G * (d / 128);   // workgroups of the kernels with their waves side by side
    if (R <= E)
        hipLaunchKernelGGL((decode_up_kernel<2, 4, 4>), dim3(G * (H / 16)), wg, 0, s, x, idx, w1, s1, h, R, E, k, d, H);
    else if (up >= kWideGroups)
        hipLaunchKernelGGL((decode_up_wide_kernel<2, 4>), dim3(up), wg, 0, s, x, idx, w1, s1, h, R, E, k, d, H);
    else
        hipLaunchKernelGGL((decode_up_kernel<4, 16, 1>), dim3(G * (H / 32)), wg, 0, s, x, idx, w1, s1, h, R, E, k, d, H);
    if (2 * R <= E) {
        if (T * (d / 32) >= 256)
            hipLaunchKernelGGL((decode_down_token_kernel<2, 4>), dim3(T * (d / 32)), dim3(1024), 0, s, h, idx, gate, w2,
                               s2, y, E, k, d, H);
        else
            hipLaunchKernelGGL((decode_down_token_kernel<1, 4>), dim3(T * (d / 16)), dim3(1024), 0, s, h, idx, gate, w2,
                               s2, y, E, k, d, H);
        return hipGetLastError();
    }
    if (down >= kWideGroups)
        hipLaunchKernelGGL((decode_down_wide_kernel<2, 2>), dim3(down), wg, 0, s, h, idx, w2, s2, ye, R, E, d, H);
    else if (R <= E)
        hipLaunchKernelGGL((decode_down_kernel<2, 4, 4>), dim3(G * (d / 32)), wg, 0, s, h, idx, w2, s2, ye, R, E, d, H);
    else
        hipLaunchKernelGGL((decode_down_kernel<4, 16, 1>), dim3(G * (d / 64)), wg, 0, s, h, idx, w2, s2, ye, R, E, d, H);
    const dim3 cg((d / 4 + 255) / 256, T), cb(256);
    if (k <= 4) hipLaunchKernelGGL(decode_combine_kernel<4>, cg, cb, 0, s, ye, idx, gate, y, E, k, d);
    else if (k <= 8) hipLaunchKernelGGL(decode_combine_kernel<8>, cg, cb, 0, s, ye, idx, gate, y, E, k, d);
    else hipLaunchKernelGGL(decode_combine_kernel<kMaxTopK>, cg, cb, 0, s, ye, idx, gate, y, E, k, d);
    return hipGetLastError();
}

}  // namespace moe
