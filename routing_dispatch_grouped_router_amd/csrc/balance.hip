// Router balance loss with the per-expert counts, and its gradient for the
// logits, for gfx950.
//
// Over the N live tokens (mask nonzero), p = softmax of a token's E logits,
// lse its log-sum-exp, f_e = counts[e] / (N k):
//   balance = E sum_e f_e P_e, P_e = (1 / N) sum_t p_te   (the Switch form the
//   router statistics use, the counts taken as constants),
//   z = (1 / N) sum_t lse_t^2,
//   dlogits[t][e] = (p_te / N) (g0 E (f_e - sum_j f_j p_tj) + 2 g1 lse_t)
// with (g0, g1) the loss's gradient for the two; rows that are not live get 0.
//
// A token's logits are read once by a group of G lanes in each direction
// (softmax statistics by cross-lane reductions in registers).  The forward
// sums probabilities per workgroup, the second launch adds the workgroups'
// partial sums; every sum runs in a fixed order and the counts are integers,
// so the results are reproducible bit for bit.
#include <algorithm>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kBalBlocks = 512;   // partial rows: two workgroups per compute unit

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int m = G / 2; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int m = G / 2; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
    return v;
}

// The V logits of this lane (experts r + G v, -inf past E), then their
// softmax and log-sum-exp over the group.  A row without a finite logit has
// no distribution: p = 0, lse = 0.
template <int G, int V>
__device__ __forceinline__ void row_softmax(const float (&l)[V], float (&p)[V], float& lse) {
    float mx = l[0];
#pragma unroll
    for (int v = 1; v < V; ++v) mx = fmaxf(mx, l[v]);
    mx = group_max<G>(mx);
    const bool none = mx == -INFINITY;
    float z = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        p[v] = none ? 0.f : expf(l[v] - mx);
        z += p[v];
    }
    z = group_sum<G>(z);
    const float inv = none ? 0.f : 1.0f / z;
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] *= inv;
    lse = none ? 0.f : mx + logf(z);
}

template <int G, int V>
__device__ __forceinline__ void load_logits(const float* logits, size_t t, int E, int r, float (&l)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = r + G * v;
        l[v] = logits[t * E + min(e, E - 1)];
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (r + G * v >= E) l[v] = -INFINITY;
}

}  // namespace

// Workgroup b takes the tokens [b rows, (b + 1) rows), 256 / G at a time.
// part: psum [nblk][E], then z [nblk]; cnt: [nblk][E], then live [nblk].
template <int G, int V>
__global__ __launch_bounds__(256) void balance_partial_kernel(const float* __restrict__ logits,
                                                              const int32_t* __restrict__ idx,
                                                              const uint8_t* __restrict__ mask, int T, int E, int k,
                                                              int rows, float* __restrict__ part,
                                                              int32_t* __restrict__ cnt) {
    constexpr int TA = 256 / G;
    __shared__ int32_t s_cnt[kMaxExperts + 1];
    __shared__ float s_p[256 * V];
    __shared__ float s_z[TA];
    const int tid = threadIdx.x, r = tid % G, grp = tid / G, nblk = gridDim.x;
    for (int i = tid; i <= E; i += 256) s_cnt[i] = 0;
    __syncthreads();
    const int t0 = blockIdx.x * rows, t1 = min(T, t0 + rows);
    float ps[V], zs = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) ps[v] = 0.f;
    int live_n = 0;
    for (int tb = t0; tb < t1; tb += TA) {
        const int t = tb + grp;
        const bool live = t < t1 && (mask == nullptr || mask[min(t, T - 1)] != 0);
        float l[V], p[V], lse;
        load_logits<G, V>(logits, (size_t)min(t, T - 1), E, r, l);
        row_softmax<G, V>(l, p, lse);
        if (live) {
#pragma unroll
            for (int v = 0; v < V; ++v) ps[v] += p[v];
            zs = fmaf(lse, lse, zs);
            ++live_n;
        }
    }
    // the tokens' choices: an index outside [0, E) is no choice
    const size_t i1 = (size_t)t1 * k;
    for (size_t i = (size_t)t0 * k + tid; i < i1; i += 256) {
        const int e = idx[i];
        if (e >= 0 && e < E && (mask == nullptr || mask[i / k] != 0)) atomicAdd(&s_cnt[e], 1);
    }
    if (r == 0) {
        s_z[grp] = zs;
        atomicAdd(&s_cnt[E], live_n);
    }
    // s_p[grp][v][r]: this group's probabilities of expert r + G v
#pragma unroll
    for (int v = 0; v < V; ++v) s_p[(grp * V + v) * G + r] = ps[v];
    __syncthreads();
    for (int e = tid; e < E; e += 256) {
        float s = 0.f;
        for (int g = 0; g < TA; ++g) s += s_p[g * V * G + e];
        part[(size_t)blockIdx.x * E + e] = s;
        cnt[(size_t)blockIdx.x * E + e] = s_cnt[e];
    }
    if (tid == 0) {
        float z = 0.f;
        for (int g = 0; g < TA; ++g) z += s_z[g];
        part[(size_t)nblk * E + blockIdx.x] = z;
        cnt[(size_t)nblk * E + blockIdx.x] = s_cnt[E];
    }
}

// counts[E + 1] (the last one the live tokens) and loss[2] from the partial
// sums: thread (e, c) adds expert e's over a chunk c of workgroups.
__global__ __launch_bounds__(1024) void balance_finish_kernel(const float* __restrict__ part,
                                                              const int32_t* __restrict__ cnt, int nblk, int E, int k,
                                                              int32_t* __restrict__ counts, float* __restrict__ loss) {
    __shared__ float s_p[1024];
    __shared__ int32_t s_c[1024];
    __shared__ float s_z[16];
    __shared__ int32_t s_n[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // z and the live tokens: one wave each takes its share of the workgroups
    float z = 0.f;
    int n = 0;
    for (int b = tid; b < nblk; b += 1024) {
        z += part[(size_t)nblk * E + b];
        n += cnt[(size_t)nblk * E + b];
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
        z += __shfl_xor(z, m);
        n += __shfl_xor(n, m);
    }
    if (lane == 0) {
        s_z[wave] = z;
        s_n[wave] = n;
    }
    const int NC = max(1, min(1024 / E, nblk)), CS = (nblk + NC - 1) / NC;
    const int e = tid % E, c = tid / E;
    float p = 0.f;
    int q = 0;
    if (c < NC) {
        constexpr int kB = 8;
        const int b0 = c * CS, b1 = min(nblk, b0 + CS);
        for (int b = b0; b < b1; b += kB) {
            float pv[kB];
            int qv[kB];
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                pv[u] = b + u < b1 ? part[(size_t)(b + u) * E + e] : 0.f;
                qv[u] = b + u < b1 ? cnt[(size_t)(b + u) * E + e] : 0;
            }
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                p += pv[u];
                q += qv[u];
            }
        }
    }
    s_p[tid] = p;
    s_c[tid] = q;
    __syncthreads();
    z = 0.f;
    n = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        z += s_z[w];
        n += s_n[w];
    }
    const float inv = n > 0 ? 1.0f / (float)n : 0.f;
    float fp = 0.f;
    if (tid < E) {
        for (int cc = 1; cc < NC; ++cc) {
            p += s_p[cc * E + tid];
            q += s_c[cc * E + tid];
        }
        counts[tid] = q;
        fp = ((float)q * inv / (float)k) * (p * inv);
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) fp += __shfl_xor(fp, m);
    __syncthreads();
    if (lane == 0) s_z[wave] = fp;
    __syncthreads();
    if (tid == 0) {
        fp = 0.f;
        for (int w = 0; w < 16; ++w) fp += s_z[w];
        counts[E] = n;
        loss[0] = (float)E * fp;
        loss[1] = z * inv;
    }
}

template <int G, int V>
__global__ __launch_bounds__(256) void balance_bwd_kernel(const float* __restrict__ logits,
                                                          const uint8_t* __restrict__ mask,
                                                          const int32_t* __restrict__ counts,
                                                          const float* __restrict__ dloss, int T, int E, int k,
                                                          int rows, float* __restrict__ dlogits) {
    constexpr int TA = 256 / G;
    const int r = threadIdx.x % G, grp = threadIdx.x / G;
    const int n = counts[E];
    const float inv = n > 0 ? 1.0f / (float)n : 0.f;
    const float gb = dloss[0] * (float)E * inv, gz = dloss[1] * 2.0f * inv;
    float f[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        f[v] = r + G * v < E ? (float)counts[min(r + G * v, E - 1)] * inv / (float)k : 0.f;
    const int t0 = blockIdx.x * rows, t1 = min(T, t0 + rows);
    for (int tb = t0; tb < t1; tb += TA) {
        const int t = tb + grp, tc = min(t, T - 1);
        const bool live = mask == nullptr || mask[tc] != 0;
        float l[V], p[V], lse;
        load_logits<G, V>(logits, (size_t)tc, E, r, l);
        row_softmax<G, V>(l, p, lse);
        float fp = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) fp = fmaf(f[v], p[v], fp);
        fp = group_sum<G>(fp);
        if (t >= t1) continue;   // whole groups
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (r + G * v < E)
                dlogits[(size_t)t * E + r + G * v] = live ? p[v] * fmaf(gb, f[v] - fp, gz * lse) : 0.f;
    }
}

namespace {

// Lanes per token: the smallest power of two G <= 64 with E / G <= 4
// (V = 4 logits a lane; at E > 256 all 64 lanes hold up to 16).
int balance_lanes(int E) {
    int G = 1;
    while (G < 64 && (E + G - 1) / G > 4) G <<= 1;
    return G;
}

// Tokens per workgroup: a multiple of those it takes at a time.
int balance_rows(int T, int E) {
    const int TA = 256 / balance_lanes(E);
    const int per = (T + kBalBlocks - 1) / kBalBlocks;
    return (per + TA - 1) / TA * TA;
}

template <int G, int V>
void partial_t(const float* logits, const int32_t* idx, const uint8_t* mask, int T, int E, int k, float* part,
               int32_t* cnt, hipStream_t s) {
    const int rows = balance_rows(T, E);
    hipLaunchKernelGGL((balance_partial_kernel<G, V>), dim3((T + rows - 1) / rows), dim3(256), 0, s, logits, idx,
                       mask, T, E, k, rows, part, cnt);
}

template <int G, int V>
void bwd_t(const float* logits, const uint8_t* mask, const int32_t* counts, const float* dloss, int T, int E, int k,
           float* dlogits, hipStream_t s) {
    const int rows = balance_rows(T, E);
    hipLaunchKernelGGL((balance_bwd_kernel<G, V>), dim3((T + rows - 1) / rows), dim3(256), 0, s, logits, mask, counts,
                       dloss, T, E, k, rows, dlogits);
}

}  // namespace

int balance_blocks(int T, int E) {
    const int rows = balance_rows(T, E);
    return (T + rows - 1) / rows;
}

hipError_t launch_balance(const float* logits, const int32_t* idx, const uint8_t* mask, int T, int E, int k,
                          int32_t* counts, float* loss, float* part, int32_t* cnt, hipStream_t s) {
    switch (balance_lanes(E)) {
        case 1: partial_t<1, 4>(logits, idx, mask, T, E, k, part, cnt, s); break;
        case 2: partial_t<2, 4>(logits, idx, mask, T, E, k, part, cnt, s); break;
        case 4: partial_t<4, 4>(logits, idx, mask, T, E, k, part, cnt, s); break;
        case 8: partial_t<8, 4>(logits, idx, mask, T, E, k, part, cnt, s); break;
        case 16: partial_t<16, 4>(logits, idx, mask, T, E, k, part, cnt, s); break;
        case 32: partial_t<32, 4>(logits, idx, mask, T, E, k, part, cnt, s); break;
        default:
            if (E <= 256) partial_t<64, 4>(logits, idx, mask, T, E, k, part, cnt, s);
            else partial_t<64, 16>(logits, idx, mask, T, E, k, part, cnt, s);
    }
    hipLaunchKernelGGL(balance_finish_kernel, dim3(1), dim3(1024), 0, s, part, cnt, balance_blocks(T, E), E, k, counts,
                       loss);
    return hipGetLastError();
}

hipError_t launch_balance_bwd(const float* logits, const uint8_t* mask, const int32_t* counts, const float* dloss,
                              int T, int E, int k, float* dlogits, hipStream_t s) {
    switch (balance_lanes(E)) {
        case 1: bwd_t<1, 4>(logits, mask, counts, dloss, T, E, k, dlogits, s); break;
        case 2: bwd_t<2, 4>(logits, mask, counts, dloss, T, E, k, dlogits, s); break;
        case 4: bwd_t<4, 4>(logits, mask, counts, dloss, T, E, k, dlogits, s); break;
        case 8: bwd_t<8, 4>(logits, mask, counts, dloss, T, E, k, dlogits, s); break;
        case 16: bwd_t<16, 4>(logits, mask, counts, dloss, T, E, k, dlogits, s); break;
        case 32: bwd_t<32, 4>(logits, mask, counts, dloss, T, E, k, dlogits, s); break;
        default:
            if (E <= 256) bwd_t<64, 4>(logits, mask, counts, dloss, T, E, k, dlogits, s);
            else bwd_t<64, 16>(logits, mask, counts, dloss, T, E, k, dlogits, s);
    }
    return hipGetLastError();
}

}  // namespace moe
