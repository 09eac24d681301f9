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
// the activations stay bfloat16.  A lane's 16-byte load is one scale block
// (32 k of one row); the four MFMAs that consume it take k in the order the
// lanes hold it, for both operands alike.  Rows are not sorted or moved: a
// workgroup finds its expert's rows in topk_idx itself, and an index outside
// [0, E) is a slot not in use.
#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kMaxRows = kDecodeTokens * kMaxTopK;

__device__ __forceinline__ float e8m0_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight E2M1 codes times 2^(byte - 127) as bfloat16 (exact).
__device__ __forceinline__ bf16x8 fp4_to_bf16(uint32_t w, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    return (bf16x8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The routed rows of group g: with R <= E a group per routed row, whose rows
// are those of its expert if it is the expert's first row (none otherwise);
// else a group per expert.  rows[0, n) in ascending order; returns n, the
// same on every thread of the workgroup's 256.
__device__ __forceinline__ int group_rows(const int32_t* idx, int R, int E, int g, int& expert, int32_t* rows,
                                          int32_t* wcnt) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    expert = R <= E ? idx[g] : g;
    if (expert < 0 || expert >= E) return 0;   // uniform
    int n = 0;
    for (int base = 0; base < R; base += 256) {
        const int r = base + tid;
        const bool mine = r < R && idx[r] == expert;
        const uint64_t b = __ballot(mine);
        if (lane == 0) wcnt[wave] = __popcll(b);
        __syncthreads();
        int off = n, all = n;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w < wave) off += wcnt[w];
            all += wcnt[w];
        }
        if (mine) rows[off + __popcll(b & ((1ull << lane) - 1ull))] = r;
        n = all;
        __syncthreads();   // wcnt is rewritten by the next 256 rows; rows[] is complete after the last
    }
    if (R <= E && rows[0] != g) return 0;      // uniform: another row of this expert comes first
    return n;
}

// NB blocks of 16 weight rows (row0[b] their first row's codes, srow0[b] its
// scales) times 16 routed rows (lane l: row l % 16 at xrow, zero unless live),
// over the 128-wide slices [s0, s1) of K.
template <int NB>
__device__ __forceinline__ void mma_slices(const uint8_t* const (&wrow)[NB], const uint8_t* const (&srow)[NB],
                                           const uint16_t* xrow, bool live, int s0, int s1, f32x4 (&acc)[NB]) {
    const int q = (threadIdx.x & 63) >> 4;
    constexpr int U = 2;   // slices in flight
    for (int s = s0; s < s1; s += U) {
        u32x4 w[U][NB], xv[U][4];
        uint32_t sc[U][NB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int sl = min(s + u, s1 - 1);   // a clamped slice is loaded, not used
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                w[u][b] = *reinterpret_cast<const u32x4*>(wrow[b] + 64 * sl + 16 * q);
                sc[u][b] = srow[b][4 * sl + q];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) xv[u][i] = *reinterpret_cast<const u32x4*>(xrow + 128 * sl + 32 * q + 8 * i);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= s1) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bf16x8 x = __builtin_bit_cast(bf16x8, live ? xv[u][i] : (u32x4){0u, 0u, 0u, 0u});
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp4_to_bf16(w[u][b][i], e8m0_scale(sc[u][b])), x,
                                                                     acc[b], 0, 0, 0);
            }
        }
    }
}

}  // namespace

// Gate and up projections: workgroup = (group, 16 hidden units).  Its four
// waves take the quarters of d; wave 0 adds them in order and stores
// h = silu(a) b, bfloat16, at h[r][H].
__global__ __launch_bounds__(256) void decode_up_kernel(const uint16_t* __restrict__ x,
                                                        const int32_t* __restrict__ idx,
                                                        const uint8_t* __restrict__ w1,
                                                        const uint8_t* __restrict__ s1, uint16_t* __restrict__ h,
                                                        int R, int E, int k, int d, int H) {
    __shared__ int32_t s_rows[kMaxRows];
    __shared__ int32_t s_cnt[4];
    __shared__ f32x4 red[4][2][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, q = lane >> 4;
    const int nb = H / 16, g = blockIdx.x / nb, hb = blockIdx.x - g * nb;
    int e;
    const int n = group_rows(idx, R, E, g, e, s_rows, s_cnt);
    if (n == 0) return;
    // packed rows of hidden units 16 hb .. + 16: gate at 64 (hb / 2) + 16 (hb % 2), up 32 further
    const size_t row = (size_t)e * 2 * H + 64 * (hb >> 1) + 16 * (hb & 1) + m;
    const uint8_t* const wrow[2] = {w1 + row * (d / 2), w1 + (row + 32) * (d / 2)};
    const uint8_t* const srow[2] = {s1 + row * (d / 32), s1 + (row + 32) * (d / 32)};
    const int ns = d / 128, sl0 = wave * ns / 4, sl1 = (wave + 1) * ns / 4;
    for (int n0 = 0; n0 < n; n0 += 16) {
        const bool live = n0 + m < n;
        const int r = s_rows[min(n0 + m, n - 1)];
        f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        mma_slices<2>(wrow, srow, x + (size_t)(r / k) * d, live, sl0, sl1, acc);
        red[wave][0][lane] = acc[0];
        red[wave][1][lane] = acc[1];
        __syncthreads();
        if (wave == 0 && live) {
            const f32x4 a = ((red[0][0][lane] + red[1][0][lane]) + red[2][0][lane]) + red[3][0][lane];
            const f32x4 b = ((red[0][1][lane] + red[1][1][lane]) + red[2][1][lane]) + red[3][1][lane];
            float o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = a[i] / (1.0f + expf(-a[i])) * b[i];
            *reinterpret_cast<uint2*>(h + (size_t)r * H + 16 * hb + 4 * q) =
                make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
        }
        __syncthreads();   // red is rewritten for the next rows
    }
}

// Down projection: workgroup = (group, 32 outputs), ye[r][d] in float32.
__global__ __launch_bounds__(256) void decode_down_kernel(const uint16_t* __restrict__ h,
                                                          const int32_t* __restrict__ idx,
                                                          const uint8_t* __restrict__ w2,
                                                          const uint8_t* __restrict__ s2, float* __restrict__ ye,
                                                          int R, int E, int d, int H) {
    __shared__ int32_t s_rows[kMaxRows];
    __shared__ int32_t s_cnt[4];
    __shared__ f32x4 red[4][2][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, q = lane >> 4;
    const int nb = d / 32, g = blockIdx.x / nb, cb = blockIdx.x - g * nb;
    int e;
    const int n = group_rows(idx, R, E, g, e, s_rows, s_cnt);
    if (n == 0) return;
    const size_t row = (size_t)e * d + 32 * cb + m;
    const uint8_t* const wrow[2] = {w2 + row * (H / 2), w2 + (row + 16) * (H / 2)};
    const uint8_t* const srow[2] = {s2 + row * (H / 32), s2 + (row + 16) * (H / 32)};
    const int ns = H / 128, sl0 = wave * ns / 4, sl1 = (wave + 1) * ns / 4;
    for (int n0 = 0; n0 < n; n0 += 16) {
        const bool live = n0 + m < n;
        const int r = s_rows[min(n0 + m, n - 1)];
        f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        mma_slices<2>(wrow, srow, h + (size_t)r * H, live, sl0, sl1, acc);
        red[wave][0][lane] = acc[0];
        red[wave][1][lane] = acc[1];
        __syncthreads();
        if (wave < 2 && live)   // wave b stores block b's outputs 32 cb + 16 b + 4 q .. + 4
            *reinterpret_cast<f32x4*>(ye + (size_t)r * d + 32 * cb + 16 * wave + 4 * q) =
                ((red[0][wave][lane] + red[1][wave][lane]) + red[2][wave][lane]) + red[3][wave][lane];
        __syncthreads();
    }
}

// y[t] = sum_j gate[t][j] ye[t k + j] in slot order over the slots in use
// (float32, rounded once); four outputs per thread.
__global__ __launch_bounds__(256) void decode_combine_kernel(const float* __restrict__ ye,
                                                             const int32_t* __restrict__ idx,
                                                             const float* __restrict__ gate, uint16_t* __restrict__ y,
                                                             int E, int k, int d) {
    const int t = blockIdx.y, c = 4 * (blockIdx.x * 256 + threadIdx.x);
    if (c >= d) return;
    f32x4 v[kMaxTopK];
    float g[kMaxTopK];
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
        g[j] = 0.f;
        v[j] = (f32x4){0.f, 0.f, 0.f, 0.f};
        if (j < k) {
            const int e = idx[t * k + j];
            if (e >= 0 && e < E) {
                g[j] = gate[t * k + j];
                v[j] = *reinterpret_cast<const f32x4*>(ye + ((size_t)t * k + j) * d + c);
            }
        }
    }
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j)
        if (j < k) s += g[j] * v[j];
    *reinterpret_cast<uint2*>(y + (size_t)t * d + c) = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
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
    hipLaunchKernelGGL(decode_down_kernel, dim3(G * (d / 32)), dim3(256), 0, s, h, idx, w2, s2, ye, R, E, d, H);
    hipLaunchKernelGGL(decode_combine_kernel, dim3((d / 4 + 255) / 256, T), dim3(256), 0, s, ye, idx, gate, y, E, k, d);
    return hipGetLastError();
}

}  // namespace moe
