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
// so the results are reproducible bit for bit.  Up to a few MB of logits each
// launch is a handful of memory latencies, not bandwidth, so the loads of
// kTok tokens a group, and of all a thread's partial sums, are issued together.
#include <algorithm>

#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

namespace {

// The forward takes at most a workgroup of 16 waves per compute unit (few
// partial rows for the second launch), the backward as many as it has tokens.
constexpr int kBalBlocks = 256;
constexpr int kBalThreads = 1024;
constexpr int kTok = 2;           // tokens of a group in flight

template <int G>
__device__ __forceinline__ float group_sum(float v) {
    return __uint_as_float(group_reduce<G>(__float_as_uint(v), AddF32{}));
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
    return __uint_as_float(group_reduce<G>(__float_as_uint(v), MaxF32{}));
}

// Expert of value v of lane r of a group, so that a load's lanes are side by side:
// runs of four where rows are 16 bytes aligned (16 values of a lane in a row:
// T = 8192, E = 1024, 10.8 us forward and 24.8 backward; so 10.3 and 18.5), else
// one (T = 13725, E = 277: with runs of four 10.5 and 15.8 us, so 10.1 and 13.9).
template <int G>
__device__ __forceinline__ int expert_of(int E, int r, int v) {
    return (E & 3) == 0 ? 4 * G * (v / 4) + 4 * r + v % 4 : G * v + r;
}

// The V logits of this lane (-inf past E), then their softmax and log-sum-exp
// over the group.  A row of -inf alone has no distribution: p = 0, lse = 0.
// fmaxf passes NaN over, so such a row is told by its sum, which is 0 for it
// alone: a finite or infinite maximum adds 1 or NaN, and a NaN logit NaN.
template <int G, int V>
__device__ __forceinline__ void row_softmax(const float (&l)[V], float (&p)[V], float& lse) {
    float mx = l[0];
#pragma unroll
    for (int v = 1; v < V; ++v) mx = fmaxf(mx, l[v]);
    mx = group_max<G>(mx);
    if (mx == -INFINITY) mx = 0.f;
    float z = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        p[v] = expf(l[v] - mx);
        z += p[v];
    }
    z = group_sum<G>(z);
    const float inv = z == 0.f ? 0.f : 1.0f / z;
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] *= inv;
    lse = z == 0.f ? 0.f : mx + logf(z);
}

template <int G, int V>
__device__ __forceinline__ void load_logits(const float* logits, size_t t, int E, int r, float (&l)[V]) {
    const float* row = logits + t * E;
    if ((E & 3) == 0) {   // whole runs of four, 16 bytes aligned
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            const f32x4 q = *reinterpret_cast<const f32x4*>(row + min(expert_of<G>(E, r, v), E - 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) l[v + i] = q[i];
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) l[v] = row[min(expert_of<G>(E, r, v), E - 1)];
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (expert_of<G>(E, r, v) >= E) l[v] = -INFINITY;
}

}  // namespace

// Workgroup b takes the tokens [b rows, (b + 1) rows), kBalThreads / G at a time.
// part: psum [nblk][E], then z [nblk]; cnt: [nblk][E], then live [nblk].  A
// single workgroup finishes by itself: counts[E + 1] and loss[2].
template <int G, int V>
__global__ __launch_bounds__(kBalThreads) void balance_partial_kernel(const float* __restrict__ logits,
                                                                      const int32_t* __restrict__ idx,
                                                                      const uint8_t* __restrict__ mask, int T, int E,
                                                                      int k, int rows, float* __restrict__ part,
                                                                      int32_t* __restrict__ cnt,
                                                                      int32_t* __restrict__ counts,
                                                                      float* __restrict__ loss) {
    constexpr int TA = kBalThreads / G, NW = kBalThreads / 64;
    __shared__ int32_t s_cnt[kMaxExperts + 1];
    __shared__ float s_p[NW][G * V];
    __shared__ float s_z[NW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = tid % G, grp = tid / G, nblk = gridDim.x;
    for (int i = tid; i <= E; i += kBalThreads) s_cnt[i] = 0;
    __syncthreads();
    const int t0 = blockIdx.x * rows, t1 = min(T, t0 + rows);
    float ps[V], zs = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) ps[v] = 0.f;
    int live_n = 0;
    for (int tb = t0; tb < t1; tb += TA * kTok) {
        float l[kTok][V];
        bool live[kTok];
#pragma unroll
        for (int u = 0; u < kTok; ++u) {
            const int t = tb + TA * u + grp, tc = min(t, T - 1);
            live[u] = t < t1 && (mask == nullptr || mask[tc] != 0);
            load_logits<G, V>(logits, (size_t)tc, E, r, l[u]);
        }
#pragma unroll
        for (int u = 0; u < kTok; ++u) {
            float p[V], lse;
            row_softmax<G, V>(l[u], p, lse);
            if (live[u]) {
#pragma unroll
                for (int v = 0; v < V; ++v) ps[v] += p[v];
                zs = fmaf(lse, lse, zs);
                ++live_n;
            }
        }
    }
    // the tokens' choices: an index outside [0, E) is no choice
    const uint32_t nc = (uint32_t)(t1 - t0) * (uint32_t)k;
    const int32_t* choice = idx + (size_t)t0 * k;
    constexpr int kC = 4;   // of a thread in flight
    for (uint32_t i = tid; i < nc; i += kC * kBalThreads) {
        int e[kC];
        bool on[kC];
#pragma unroll
        for (int u = 0; u < kC; ++u) {
            const uint32_t j = min(i + u * kBalThreads, nc - 1);
            e[u] = choice[j];
            on[u] = i + u * kBalThreads < nc && (mask == nullptr || mask[t0 + (int)(j / (uint32_t)k)] != 0);
        }
#pragma unroll
        for (int u = 0; u < kC; ++u)
            if (on[u] && e[u] >= 0 && e[u] < E) atomicAdd(&s_cnt[e[u]], 1);
    }
    // the wave's groups, then the waves in order
    if (r != 0) {
        zs = 0.f;
        live_n = 0;
    }
#pragma unroll
    for (int i = 32; i >= G; i >>= 1) {
        zs += __shfl_xor(zs, i);
        live_n += __shfl_xor(live_n, i);
#pragma unroll
        for (int v = 0; v < V; ++v) ps[v] += __shfl_xor(ps[v], i);
    }
    if (lane < G) {
#pragma unroll
        for (int v = 0; v < V; ++v) s_p[wave][expert_of<G>(E, r, v)] = ps[v];
    }
    if (lane == 0) {
        s_z[wave] = zs;
        atomicAdd(&s_cnt[E], live_n);
    }
    __syncthreads();
    static_assert(kMaxExperts <= kBalThreads, "a thread an expert");
    const int n = s_cnt[E];
    const float inv = n > 0 ? 1.0f / (float)n : 0.f;
    float fp = 0.f;
    if (tid < E) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) s += s_p[w][tid];
        const int c = s_cnt[tid];
        if (nblk == 1) {
            counts[tid] = c;
            fp = ((float)c * inv / (float)k) * (s * inv);
        } else {
            part[(size_t)blockIdx.x * E + tid] = s;
            cnt[(size_t)blockIdx.x * E + tid] = c;
        }
    }
    float z = 0.f;
    if (tid == 0) {
#pragma unroll
        for (int w = 0; w < NW; ++w) z += s_z[w];
    }
    if (nblk == 1) {
#pragma unroll
        for (int i = 32; i >= 1; i >>= 1) fp += __shfl_xor(fp, i);
        __syncthreads();   // s_z has been read
        if (lane == 0) s_z[wave] = fp;
        __syncthreads();
        if (tid == 0) {
            fp = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) fp += s_z[w];
            counts[E] = n;
            loss[0] = (float)E * fp;
            loss[1] = z * inv;
        }
    } else if (tid == 0) {
        part[(size_t)nblk * E + blockIdx.x] = z;
        cnt[(size_t)nblk * E + blockIdx.x] = n;
    }
}

// counts[E + 1] (the last one the live tokens) and loss[2] from the partial
// sums.  Workgroup b takes the experts [b EW, b EW + EW): thread (e, c) adds
// expert e's over a chunk c of the partial rows.  One compute unit reads the
// rows of 128 experts in a latency or two, those of 1024 in 25 us, so more
// experts go to more workgroups and their shares of the balance loss (fpart)
// to balance_sum_kernel.
constexpr int kFinishExperts = 128;

__global__ __launch_bounds__(1024) void balance_finish_kernel(const float* __restrict__ part,
                                                              const int32_t* __restrict__ cnt, int nblk, int E, int k,
                                                              int32_t* __restrict__ counts, float* __restrict__ loss,
                                                              float* __restrict__ fpart) {
    __shared__ float s_p[1024];
    __shared__ int32_t s_c[1024];
    __shared__ float s_z[16];
    __shared__ int32_t s_n[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    float z = 0.f;
    int n = 0;
    for (int b = tid; b < nblk; b += 1024) {
        z += part[(size_t)nblk * E + b];
        n += cnt[(size_t)nblk * E + b];
    }
    const int e0 = blockIdx.x * kFinishExperts, EW = min(kFinishExperts, E - e0);
    const int NC = max(1, min(1024 / EW, nblk)), CS = (nblk + NC - 1) / NC;
    const int e = tid % EW, c = tid / EW;
    float p = 0.f;
    int q = 0;
    if (c < NC) {
        constexpr int kB = 16;
        const int b0 = c * CS, b1 = min(nblk, b0 + CS);
        for (int b = b0; b < b1; b += kB) {
            float pv[kB];
            int qv[kB];
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                pv[u] = b + u < b1 ? part[(size_t)(b + u) * E + e0 + e] : 0.f;
                qv[u] = b + u < b1 ? cnt[(size_t)(b + u) * E + e0 + e] : 0;
            }
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                p += pv[u];
                q += qv[u];
            }
        }
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
    if (tid < EW) {
        for (int cc = 1; cc < NC; ++cc) {
            p += s_p[cc * EW + tid];
            q += s_c[cc * EW + tid];
        }
        counts[e0 + tid] = q;
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
        if (gridDim.x == 1) loss[0] = (float)E * fp;
        else fpart[blockIdx.x] = fp;
        if (blockIdx.x == 0) {
            counts[E] = n;
            loss[1] = z * inv;
        }
    }
}

__global__ __launch_bounds__(64) void balance_sum_kernel(const float* __restrict__ fpart, int n, int E,
                                                         float* __restrict__ loss) {
    float v = threadIdx.x < (unsigned)n ? fpart[threadIdx.x] : 0.f;
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    if (threadIdx.x == 0) loss[0] = (float)E * v;
}

// dlogits may be logits: a group reads its row before it writes it, and what the
// groups past T read of row T - 1 is not used.
template <int G, int V>
__global__ __launch_bounds__(256) void balance_bwd_kernel(const float* logits,
                                                          const uint8_t* __restrict__ mask,
                                                          const int32_t* __restrict__ counts,
                                                          const float* __restrict__ dloss, int T, int E, int k,
                                                          float* dlogits) {
    constexpr int TA = 256 / G;
    const int r = threadIdx.x % G, grp = threadIdx.x / G;
    const int n = counts[E];
    const float inv = n > 0 ? 1.0f / (float)n : 0.f;
    const float gb = dloss[0] * (float)E * inv, gz = dloss[1] * 2.0f * inv;
    float f[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        f[v] = expert_of<G>(E, r, v) < E ? (float)counts[min(expert_of<G>(E, r, v), E - 1)] * inv / (float)k : 0.f;
    const int tb = blockIdx.x * TA * kTok;
    float l[kTok][V];
    bool live[kTok];
#pragma unroll
    for (int u = 0; u < kTok; ++u) {
        const int tc = min(tb + TA * u + grp, T - 1);
        live[u] = mask == nullptr || mask[tc] != 0;
        load_logits<G, V>(logits, (size_t)tc, E, r, l[u]);
    }
#pragma unroll
    for (int u = 0; u < kTok; ++u) {
        const int t = tb + TA * u + grp;
        float p[V], lse, fp = 0.f;
        row_softmax<G, V>(l[u], p, lse);
#pragma unroll
        for (int v = 0; v < V; ++v) fp = fmaf(f[v], p[v], fp);
        fp = group_sum<G>(fp);
        if (t >= T) continue;   // whole groups
        float* row = dlogits + (size_t)t * E;
#pragma unroll
        for (int v = 0; v < V; ++v) p[v] = live[u] ? p[v] * fmaf(gb, f[v] - fp, gz * lse) : 0.f;
        if ((E & 3) == 0) {
#pragma unroll
            for (int v = 0; v < V; v += 4)
                if (expert_of<G>(E, r, v) < E)
                    *reinterpret_cast<f32x4*>(row + expert_of<G>(E, r, v)) = (f32x4){p[v], p[v + 1], p[v + 2], p[v + 3]};
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (expert_of<G>(E, r, v) < E) row[expert_of<G>(E, r, v)] = p[v];
        }
    }
}

namespace {

// Lanes per token: the smallest power of two G <= 64 with E / G <= 4
// (V = 4 logits a lane; at E > 256 all 64 lanes hold 8, or up to 16 beyond 512:
// T = 16384, E = 512, 9.7 us forward and 17 backward with 8, 13.7 and 22 with 16).
int balance_lanes(int E) {
    int G = 1;
    while (G < 64 && (E + G - 1) / G > 4) G <<= 1;
    return G;
}

// Tokens per workgroup of the forward: a multiple of those it takes at a time.
// What one workgroup reads in two batches it takes alone, which saves the second
// launch (T = 1000, E = 8, both directions: 12.4 us instead of 15.9; T = 1000,
// E = 16, k = 16: 7.6 us of kernel against 4.7 + 3.4 and the launch).
int balance_rows(int T, int E) {
    const int TA = kBalThreads / balance_lanes(E);
    if (T <= 2 * kTok * TA) return T;
    const int per = (T + kBalBlocks - 1) / kBalBlocks;
    return (per + TA - 1) / TA * TA;
}

template <int G, int V>
void partial_t(const float* logits, const int32_t* idx, const uint8_t* mask, int T, int E, int k, float* part,
               int32_t* cnt, int32_t* counts, float* loss, hipStream_t s) {
    const int rows = balance_rows(T, E);
    hipLaunchKernelGGL((balance_partial_kernel<G, V>), dim3((T + rows - 1) / rows), dim3(kBalThreads), 0, s, logits,
                       idx, mask, T, E, k, rows, part, cnt, counts, loss);
}

template <int G, int V>
void bwd_t(const float* logits, const uint8_t* mask, const int32_t* counts, const float* dloss, int T, int E, int k,
           float* dlogits, hipStream_t s) {
    constexpr int per = 256 / G * kTok;
    hipLaunchKernelGGL((balance_bwd_kernel<G, V>), dim3((T + per - 1) / per), dim3(256), 0, s, logits, mask, counts,
                       dloss, T, E, k, dlogits);
}

}  // namespace

static int balance_blocks(int T, int E) {
    const int rows = balance_rows(T, E);
    return (T + rows - 1) / rows;
}

size_t balance_part_floats(int T, int E) {
    return (size_t)balance_blocks(T, E) * (E + 1) + kMaxExperts / kFinishExperts;
}

hipError_t launch_balance(const float* logits, const int32_t* idx, const uint8_t* mask, int T, int E, int k,
                          int32_t* counts, float* loss, float* part, int32_t* cnt, hipStream_t s) {
    switch (balance_lanes(E)) {
        case 1: partial_t<1, 4>(logits, idx, mask, T, E, k, part, cnt, counts, loss, s); break;
        case 2: partial_t<2, 4>(logits, idx, mask, T, E, k, part, cnt, counts, loss, s); break;
        case 4: partial_t<4, 4>(logits, idx, mask, T, E, k, part, cnt, counts, loss, s); break;
        case 8: partial_t<8, 4>(logits, idx, mask, T, E, k, part, cnt, counts, loss, s); break;
        case 16: partial_t<16, 4>(logits, idx, mask, T, E, k, part, cnt, counts, loss, s); break;
        case 32: partial_t<32, 4>(logits, idx, mask, T, E, k, part, cnt, counts, loss, s); break;
        default:
            if (E <= 256) partial_t<64, 4>(logits, idx, mask, T, E, k, part, cnt, counts, loss, s);
            else if (E <= 512) partial_t<64, 8>(logits, idx, mask, T, E, k, part, cnt, counts, loss, s);
            else partial_t<64, 16>(logits, idx, mask, T, E, k, part, cnt, counts, loss, s);
    }
    const int nblk = balance_blocks(T, E);
    if (nblk == 1) return hipGetLastError();
    const int nf = (E + kFinishExperts - 1) / kFinishExperts;
    float* fpart = part + (size_t)nblk * (E + 1);
    hipLaunchKernelGGL(balance_finish_kernel, dim3(nf), dim3(1024), 0, s, part, cnt, nblk, E, k, counts, loss, fpart);
    if (nf > 1) hipLaunchKernelGGL(balance_sum_kernel, dim3(1), dim3(64), 0, s, fpart, nf, E, loss);
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
            else if (E <= 512) bwd_t<64, 8>(logits, mask, counts, dloss, T, E, k, dlogits, s);
            else bwd_t<64, 16>(logits, mask, counts, dloss, T, E, k, dlogits, s);
    }
    return hipGetLastError();
}

}  // namespace moe
