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
#include <algorithm>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

// Three bfloat16 terms of eight float32 values.
__device__ __forceinline__ void split3(const float (&v)[8], bf16x8 (&o)[3]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __bf16 a = (__bf16)v[i];
        const float r = v[i] - (float)a;
        const __bf16 b = (__bf16)r;
        o[0][i] = a;
        o[1][i] = b;
        o[2][i] = (__bf16)(r - (float)b);
    }
}

// c += a b for operands of TA and three terms.
template <int TA>
__device__ __forceinline__ f32x4 mfma_terms(const bf16x8 (&a)[TA], const bf16x8 (&b)[3], f32x4 c) {
#pragma unroll
    for (int i = TA - 1; i >= 0; --i)
#pragma unroll
        for (int j = 2 - i; j >= 0; --j) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], c, 0, 0, 0);
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

}  // namespace

// dx: a workgroup owns 64 tokens and 256 columns, a wave 64 of the columns.
// D = W_r dL^T as 16 x 16 blocks: M = columns, N = tokens, K = experts.  Row m
// of the wave's block mt is column 32 (mt / 2) + 8 (m / 4) + 4 (mt % 2) + m % 4,
// so that a lane's blocks 2 p and 2 p + 1 hold 8 consecutive columns of one
// token and four lanes 32: the result is read and written in 64-byte pieces.  `add`: row t of add (pos NULL), or the sum
// of its rows pos[t][0 .. k), or nothing (add NULL).
template <bool BF>
__global__ __launch_bounds__(256) void router_dx_kernel(const float* __restrict__ dL, const void* __restrict__ w,
                                                        const void* add, const int32_t* __restrict__ pos, int k,
                                                        void* dx, int T, int d, int E) {
    constexpr int TA = BF ? 1 : 3;
    constexpr int NC = BF ? 1 : 2;       // 16-byte chunks of 8 columns
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, q = lane >> 4;
    const int ncb = (d + 255) / 256, tb = blockIdx.x / ncb;
    const int t0 = tb * 64, c0 = (int)(blockIdx.x - tb * ncb) * 256 + wave * 64;
    if (c0 >= d) return;
    const bool vec = (E & 7) == 0;
    f32x4 acc[4][4];   // [column block][token block]
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + 8 * q, n = E - e;
        bf16x8 b[4][3];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
            load_terms<false>(dL, (size_t)min(t0 + 16 * nt + m, T - 1) * E + e, n, vec, b[nt]);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            bf16x8 a[TA];
            load_terms<BF>(w, (size_t)(c0 + 32 * (mt >> 1) + 8 * (m >> 2) + 4 * (mt & 1) + (m & 3)) * E + e, n, vec, a);
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) acc[mt][nt] = mfma_terms<TA>(a, b[nt], acc[mt][nt]);
        }
    }
    // 8 columns from c0 + 32 p + 8 q: NC chunks
    const size_t row_chunks = (size_t)d / (BF ? 8 : 4), cb = (size_t)(c0 + 8 * q) / (BF ? 8 : 4);
    const u32x4* src = static_cast<const u32x4*>(add);
    u32x4* dst = static_cast<u32x4*>(dx);
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
        const int t = t0 + 16 * nt + m;
        if (t >= T) continue;
        float base[2][8];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int i = 0; i < 8; ++i) base[p][i] = 0.f;
        if (src) {
            const int rows = pos ? k : 1;
            for (int j = 0; j < rows; ++j) {
                const size_t r = pos ? (size_t)pos[(size_t)t * k + j] : (size_t)t;
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int g = 0; g < NC; ++g) {
                        const u32x4 v = src[r * row_chunks + cb + 4 * NC * p + g];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (BF) {
                                base[p][2 * i] += __uint_as_float(v[i] << 16);
                                base[p][2 * i + 1] += __uint_as_float(v[i] & 0xFFFF0000u);
                            } else {
                                base[p][4 * (g % 2) + i] += __uint_as_float(v[i]);
                            }
                        }
                    }
            }
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) base[mt >> 1][4 * (mt & 1) + i] += acc[mt][nt][i];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int g = 0; g < NC; ++g) {
                u32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = BF ? pack_bf16x2(base[p][2 * i], base[p][2 * i + 1]) : __float_as_uint(base[p][4 * (g % 2) + i]);
                dst[(size_t)t * row_chunks + cb + 4 * NC * p + g] = o;
            }
    }
}

// dW_r partials: a workgroup sums 128 columns x 16 NT experts over a range of
// tokens, 32 at a time.  M = columns, N = experts, K = tokens.  The x tile is
// staged in LDS as blocks of 16 columns [32 tokens][16] (32-byte rows, blocks
// 32 bytes apart in the banks) and read transposed (ds_read_b64_tr_b16: 16
// lanes addressing rows r0 + L / 4 and columns 4 (L % 4) .. + 3 receive rows
// r0 .. r0 + 3 of column L); the dL operands are split once, by wave nt for
// experts 16 nt .. + 16, and shared through LDS.  Two buffers: the next tile's
// loads are in flight during a tile's products.
template <bool BF, int NT>
__global__ __launch_bounds__(256) void router_dw_kernel(const float* __restrict__ dL, const void* __restrict__ x,
                                                        float* __restrict__ part, int T, int d, int E, int rows) {
    typedef short v4s __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4s* lp;
    constexpr int TA = BF ? 1 : 3;
    constexpr int kTile = 32 * 32 + 32;                 // bytes of a 16-column block, padded
    constexpr int NX = BF ? 1 : 2;                      // 16-byte loads of 8 columns
    __shared__ __align__(16) char s_x[2][TA][8 * kTile];
    __shared__ u32x4 s_b[2][NT][3][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, q = lane >> 4;
    const int c0 = blockIdx.x * 128, e0 = blockIdx.y * 16 * NT;
    const int t0 = blockIdx.z * rows, t1 = min(T, t0 + rows);
    const size_t rowc = (size_t)d / (BF ? 8 : 4);       // 16-byte chunks of a row
    f32x4 acc[2][NT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};

    u32x4 xr[2][NX];
    float br[8];
    // thread item i: token tid / 16 + 16 i of the tile, columns 8 (tid % 16) .. + 8
    auto load = [&](int tb) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = tb + (tid >> 4) + 16 * i, c = c0 + 8 * (tid & 15);
#pragma unroll
            for (int g = 0; g < NX; ++g)
                xr[i][g] = t < t1 && c < d
                               ? static_cast<const u32x4*>(x)[(size_t)t * rowc + (size_t)c / (BF ? 8 : 4) + g]
                               : (u32x4){0u, 0u, 0u, 0u};
        }
        if (wave < NT) {
            const int e = e0 + 16 * wave + m;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int t = tb + 8 * q + j;
                br[j] = t < t1 && e < E ? dL[(size_t)t * E + e] : 0.f;
            }
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int tl = (tid >> 4) + 16 * i, c8 = tid & 15;
            const int off = (c8 >> 1) * kTile + tl * 32 + (c8 & 1) * 16;
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
            split3(br, o);
#pragma unroll
            for (int p = 0; p < 3; ++p) s_b[buf][wave][p][lane] = __builtin_bit_cast(u32x4, o[p]);
        }
    };

    load(t0);
    int buf = 0;
    for (int tb = t0; tb < t1; tb += 32, buf ^= 1) {
        stage(buf);
        __syncthreads();   // also: every wave has left the buffer that is written next
        if (tb + 32 < t1) load(tb + 32);
        bf16x8 a[2][TA];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int p = 0; p < TA; ++p) {
                const __attribute__((address_space(3))) char* base =
                    (const __attribute__((address_space(3))) char*)(const __attribute__((address_space(3))) void*)
                        &s_x[buf][p][(2 * wave + mt) * kTile];
                const uint32_t off = (uint32_t)(8 * q + m / 4) * 32u + (uint32_t)(m % 4) * 8u;
                const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(base + off));
                const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(base + off + 128u));
                a[mt][p] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            bf16x8 b[3];
#pragma unroll
            for (int p = 0; p < 3; ++p) b[p] = __builtin_bit_cast(bf16x8, s_b[buf][nt][p][lane]);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) acc[mt][nt] = mfma_terms<TA>(a[mt], b, acc[mt][nt]);
        }
    }
    float* dst = part + (size_t)blockIdx.z * d * E;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + 32 * wave + 16 * mt + 4 * q + i, e = e0 + 16 * nt + m;
                if (c < d && e < E) dst[(size_t)c * E + e] = acc[mt][nt][i];
            }
}

// dw[i] = sum over the S token ranges of part[.][i], in order.
__global__ __launch_bounds__(256) void router_dw_reduce_kernel(const float* __restrict__ part, int S, size_t n,
                                                               float* __restrict__ dw) {
    constexpr int kB = 8;
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
    int nt, wx, wy, rows, S;
};

RouterDwPlan router_dw_plan(int T, int d, int E) {
    RouterDwPlan p{};
    p.nt = E <= 16 ? 1 : (E <= 32 ? 2 : 4);
    p.wx = (d + 127) / 128;
    p.wy = (E + 16 * p.nt - 1) / (16 * p.nt);
    const int want = std::max(1, 512 / (p.wx * p.wy));
    const int ranges = std::max(1, std::min(want, (T + 127) / 128));
    p.rows = ((T + ranges - 1) / ranges + 31) / 32 * 32;
    p.S = (T + p.rows - 1) / p.rows;
    return p;
}

template <bool BF>
void launch_router_dw_t(const float* dL, const void* x, float* dst, const RouterDwPlan& p, int T, int d, int E,
                        hipStream_t s) {
    const dim3 g(p.wx, p.wy, p.S), b(256);
    if (p.nt == 1) hipLaunchKernelGGL((router_dw_kernel<BF, 1>), g, b, 0, s, dL, x, dst, T, d, E, p.rows);
    else if (p.nt == 2) hipLaunchKernelGGL((router_dw_kernel<BF, 2>), g, b, 0, s, dL, x, dst, T, d, E, p.rows);
    else hipLaunchKernelGGL((router_dw_kernel<BF, 4>), g, b, 0, s, dL, x, dst, T, d, E, p.rows);
}

}  // namespace

hipError_t launch_router_dx(int act, const float* dL, const void* w_router, const void* add, const int32_t* pos, int k,
                            void* dx, int T, int d, int E, hipStream_t s) {
    const dim3 g((T + 63) / 64 * ((d + 255) / 256)), b(256);
    if (act == kF32)
        hipLaunchKernelGGL((router_dx_kernel<false>), g, b, 0, s, dL, w_router, add, pos, k, dx, T, d, E);
    else
        hipLaunchKernelGGL((router_dx_kernel<true>), g, b, 0, s, dL, w_router, add, pos, k, dx, T, d, E);
    return hipGetLastError();
}

size_t router_dw_part_bytes(int T, int d, int E) {
    const RouterDwPlan p = router_dw_plan(T, d, E);
    return p.S > 1 ? (size_t)p.S * d * E * 4 : 0;
}

hipError_t launch_router_dw(int act, const float* dL, const void* x, float* part, float* dw_router, int T, int d,
                            int E, hipStream_t s) {
    const RouterDwPlan p = router_dw_plan(T, d, E);
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
