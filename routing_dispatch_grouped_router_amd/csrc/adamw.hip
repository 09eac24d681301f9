// The end of a training step over many tensors at once, for gfx950: the norm of
// all gradients, and the AdamW step.
//
//   norm = sqrt(sum over all tensors of g^2),  factor = max_norm / norm if norm > max_norm, else 1
//   t = steps taken + 1,  g' = factor g,
//   m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2,
//   w = w - lr (m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps) + decay w).
//
// One launch for all tensors of a kind: a table in device memory says where they
// are, a workgroup takes chunks of 4096 elements, eight consecutive ones a
// thread, so that every stream moves in 16-byte pieces.  Elements past a
// tensor's last multiple of eight go one by one; nothing outside a tensor is
// touched.
//
// Moments in 8 bits: m and r = sqrt(v) as E4M3 codes times a float32 scale,
// amax / 448, for each 128 elements (the root halves the range that the codes
// have to cover).  Rounded to nearest, v would stand still: a step moves it by
// (1 - b2)(g^2 - v), a thousandth of it, and its codes are a sixteenth apart.
// So the codes are rounded stochastically, up with the probability that the
// remainder says, which keeps the moments right on average; likewise bfloat16
// weights without a float32 master, whose last bit is larger than most steps.
// The random bits are a hash of (seed, step, tensor, block, element): steps are
// reproducible bit for bit.
// A root that is right on average has a square too large by the rounding's
// variance.  A step leaves r close to the code it came from, a part f of the way to
// the next that is in proportion to 1 - b2, and the variance f (1 - f) with it: v
// is larger by 3 to 4 % on average whatever b2 is (gradients of a normal
// distribution, b2 from 0.95 to 0.999), its root by half of that.
//
// HBM bounds it: an element's 30 bytes (bf16 weight, float32 master, moments and
// gradient), 28 (float32) or 12 (bf16 alone, 8-bit moments) are read and
// written once.
#include <algorithm>

#include "moe_device.h"
#include "moe_internal.h"
#include "params.h"

namespace moe {

namespace {

// ----------------------------------------------------------------------------- eight elements of a stream

// Elements [i, i + 8) below n of p as float32 (zero from n on).
__device__ __forceinline__ void load8(const float* p, uint64_t i, uint64_t n, float (&v)[8]) {
    if (i + 8 <= n) {
        const u32x4 a = *reinterpret_cast<const u32x4*>(p + i), b = *reinterpret_cast<const u32x4*>(p + i + 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = __uint_as_float(a[k]);
            v[4 + k] = __uint_as_float(b[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = i + k < n ? p[i + k] : 0.f;
    }
}
__device__ __forceinline__ void load8(const uint16_t* p, uint64_t i, uint64_t n, float (&v)[8]) {
    if (i + 8 <= n) {
        unpack16<true>(*reinterpret_cast<const u32x4*>(p + i), v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = i + k < n ? bf16_to_f32(p[i + k]) : 0.f;
    }
}
__device__ __forceinline__ void store8(float* p, uint64_t i, uint64_t n, const float (&v)[8]) {
    if (i + 8 <= n) {
        u32x4 a, b;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            a[k] = __float_as_uint(v[k]);
            b[k] = __float_as_uint(v[4 + k]);
        }
        *reinterpret_cast<u32x4*>(p + i) = a;
        *reinterpret_cast<u32x4*>(p + i + 4) = b;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + k < n) p[i + k] = v[k];
    }
}
__device__ __forceinline__ void store8(uint16_t* p, uint64_t i, uint64_t n, const float (&v)[8]) {
    if (i + 8 <= n) {
        *reinterpret_cast<u32x4*>(p + i) = pack16<true>(v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + k < n) p[i + k] = f32_to_bf16(v[k]);
    }
}

// ----------------------------------------------------------------------------- random bits

// The 32-bit finalizer of MurmurHash3 (A. Appleby, public domain).
__device__ __forceinline__ uint32_t mix(uint32_t h) {
    h = (h ^ (h >> 16)) * 0x85EBCA6Bu;
    h = (h ^ (h >> 13)) * 0xC2B2AE35u;
    return h ^ (h >> 16);
}

// ----------------------------------------------------------------------------- 8-bit moments

// Eight codes times their scale (zero from n on).
__device__ __forceinline__ void load_codes(const uint8_t* p, uint64_t i, uint64_t n, float scale, float (&v)[8]) {
    uint32_t w[2] = {0u, 0u};
    if (i + 8 <= n) {
        const uint2 a = *reinterpret_cast<const uint2*>(p + i);
        w[0] = a.x;
        w[1] = a.y;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + k < n) w[k / 4] |= (uint32_t)p[i + k] << (8 * (k % 4));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[k], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[k], true);
        v[4 * k] = a[0] * scale;
        v[4 * k + 1] = a[1] * scale;
        v[4 * k + 2] = b[0] * scale;
        v[4 * k + 3] = b[1] * scale;
    }
}

// Codes of eight values of a block and the block's scale; the 16 lanes that hold
// a block call it together.  r16: their random bits.  A value's exponent and
// fraction as E4M3 has them stand above 20 further bits once it is times 2^-120:
// 20 random bits (16 and a half) are added there and the sum cut.  Infinite and
// NaN values get the NaN code and do not count for the scale; a block below
// 2^-100 is zero.
__device__ __forceinline__ void store_codes(uint8_t* p, float* scales, uint64_t i, uint64_t n, const float (&v)[8],
                                            const uint32_t (&r16)[8]) {
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float a = fabsf(v[k]);
        amax = fmaxf(amax, a < INFINITY ? a : 0.f);
    }
    amax = __uint_as_float(group_reduce<16>(__float_as_uint(amax), MaxF32()));
    if (amax < 0x1p-100f) amax = 0.f;
    if (i % kParamBlock == 0 && i < n) scales[i / kParamBlock] = amax / 448.f;
    const float inv = amax > 0.f ? 448.f / amax : 0.f;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t u = __float_as_uint(fminf(fabsf(v[k]) * inv, 448.f) * 0x1p-120f);
        uint32_t c = min((u + (r16[k] * 16 + 8)) >> 20, 0x7Eu);
        if (!(fabsf(v[k]) < INFINITY)) c = 0x7F;
        w[k / 4] |= (c | (v[k] < 0.f ? 0x80u : 0u)) << (8 * (k % 4));
    }
    if (i + 8 <= n) {
        *reinterpret_cast<uint2*>(p + i) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + k < n) p[i + k] = (uint8_t)(w[k / 4] >> (8 * (k % 4)));
    }
}

// ----------------------------------------------------------------------------- the step

// beta^t by squaring (t >= 1).
__device__ __forceinline__ double power(double beta, uint32_t t) {
    double p = 1.0;
    for (; t; t >>= 1, beta *= beta)
        if (t & 1) p *= beta;
    return p;
}

struct StepScalars {
    float factor, lr, c1, c2_root, b1, g1, b2, g2, eps;   // c1 = 1 / (1 - b1^t), c2_root = 1 / sqrt(1 - b2^t)
    uint32_t key;
};

// One chunk.  W: weights float32 (0), bfloat16 with a master (1), bfloat16 alone (2).
template <int W, bool S8, typename G>
__device__ __forceinline__ void adamw_chunk(const ParamDesc& d, uint64_t base, const StepScalars& s) {
    const float lr = s.lr * d.lr_scale;
    const uint32_t key = S8 || W == 2 ? mix(s.key + d.index) : 0u;
#pragma unroll
    for (int u = 0; u < kParamChunk / 2048; ++u) {
        const uint64_t i = base + 2048 * u + 8 * threadIdx.x;
        float g[8], w[8], m[8], v[8];
        load8(static_cast<const G*>(d.g), i, d.n, g);
        if (W == 0) load8(static_cast<const float*>(d.w), i, d.n, w);
        else if (W == 1) load8(d.master, i, d.n, w);
        else load8(static_cast<const uint16_t*>(d.w), i, d.n, w);
        if (S8) {
            load_codes(static_cast<const uint8_t*>(d.m), i, d.n, i < d.n ? d.m_scale[i / kParamBlock] : 0.f, m);
            load_codes(static_cast<const uint8_t*>(d.v), i, d.n, i < d.n ? d.v_scale[i / kParamBlock] : 0.f, v);
        } else {
            load8(static_cast<const float*>(d.m), i, d.n, m);
            load8(static_cast<const float*>(d.v), i, d.n, v);
        }
        float r[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float gk = g[k] * s.factor;
            m[k] = fmaf(s.b1, m[k], s.g1 * gk);
            v[k] = fmaf(s.b2, S8 ? v[k] * v[k] : v[k], s.g2 * gk * gk);
            r[k] = sqrtf(v[k]);
            const float step = m[k] * s.c1 / fmaf(r[k], s.c2_root, s.eps);
            w[k] = fmaf(-lr, fmaf(d.decay, w[k], step), w[k]);
        }
        uint32_t h[8];
        if (S8 || W == 2) {
            const uint32_t kb = mix(key ^ (uint32_t)(i / kParamBlock));
#pragma unroll
            for (int k = 0; k < 8; ++k) h[k] = mix(kb + ((uint32_t)(i % kParamBlock) + k) * 0x9E3779B9u);
        }
        if (S8) {
            uint32_t lo[8], hi[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                lo[k] = h[k] & 0xFFFFu;
                hi[k] = h[k] >> 16;
            }
            store_codes(static_cast<uint8_t*>(d.m), d.m_scale, i, d.n, m, lo);
            store_codes(static_cast<uint8_t*>(d.v), d.v_scale, i, d.n, r, hi);
        } else {
            store8(static_cast<float*>(d.m), i, d.n, m);
            store8(static_cast<float*>(d.v), i, d.n, v);
        }
        if (W == 0) {
            store8(static_cast<float*>(d.w), i, d.n, w);
        } else {
            if (W == 1) {
                store8(d.master, i, d.n, w);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t b = __float_as_uint(w[k]), up = b + (mix(h[k] + 0x7F4A7C15u) & 0xFFFFu);
                    if (fabsf(w[k]) < INFINITY) w[k] = __uint_as_float(up & 0xFFFF0000u);
                }
            }
            store8(static_cast<uint16_t*>(d.w), i, d.n, w);
        }
    }
}

template <int W, bool S8, typename G>
__global__ __launch_bounds__(256) void adamw_kernel(AdamArgs a) {
    const ParamDesc* descs = reinterpret_cast<const ParamDesc*>(a.table + a.descs);
    const uint32_t* map = reinterpret_cast<const uint32_t*>(a.table + a.map);
    const int32_t taken = *reinterpret_cast<const volatile int32_t*>(a.step);
    const float factor = a.clip ? a.clip[1] : 1.f;
    const bool finite = fabsf(factor) < INFINITY;
    if (finite) {   // else the step is left out: the gradients' norm was infinite or NaN
        const uint32_t t = (uint32_t)taken + 1u;
        StepScalars s;
        s.factor = factor;
        s.lr = *a.lr;
        s.c1 = (float)(1.0 / (1.0 - power(a.beta1, t)));
        s.c2_root = (float)(1.0 / sqrt(1.0 - power(a.beta2, t)));
        s.b1 = (float)a.beta1;
        s.g1 = (float)(1.0 - a.beta1);
        s.b2 = (float)a.beta2;
        s.g2 = (float)(1.0 - a.beta2);
        s.eps = a.eps;
        s.key = mix(mix(t) ^ a.seed);
        for (int c = a.first + blockIdx.x; c < a.end; c += gridDim.x) {
            const ParamDesc d = descs[map[c]];
            adamw_chunk<W, S8, G>(d, (uint64_t)(c - (int)d.first) * kParamChunk, s);
        }
    }
    if (!a.count) return;
    __syncthreads();   // every wave has read the count
    if (threadIdx.x == 0) {
        // the last workgroup to come here counts the step: every other one has read the count
        uint32_t* ticket = reinterpret_cast<uint32_t*>(a.step + 1);
        if (atomicInc(ticket, gridDim.x - 1) == gridDim.x - 1 && finite) a.step[0] = taken + 1;
    }
}

// ----------------------------------------------------------------------------- the norm

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return ((red[0] + red[1]) + red[2]) + red[3];
}

// Squares summed in float64 (no float32 value's square leaves its range), a
// workgroup's chunks in order, the workgroups' sums in order by the last of them.
__global__ __launch_bounds__(256) void grad_norm_kernel(unsigned char* table, size_t descs_at, size_t map_at,
                                                        int chunks, float max_norm, float* __restrict__ out) {
    __shared__ double red[4];
    __shared__ bool last;
    ParamHead* head = reinterpret_cast<ParamHead*>(table);
    const ParamDesc* descs = reinterpret_cast<const ParamDesc*>(table + descs_at);
    const uint32_t* map = reinterpret_cast<const uint32_t*>(table + map_at);
    double sum = 0.0;
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const ParamDesc d = descs[map[c]];
        const uint64_t base = (uint64_t)(c - (int)d.first) * kParamChunk;
        float g[kParamChunk / 2048][8];
#pragma unroll
        for (int u = 0; u < kParamChunk / 2048; ++u) {
            const uint64_t i = base + 2048 * u + 8 * threadIdx.x;
            if (d.g_bf16) load8(static_cast<const uint16_t*>(d.g), i, d.n, g[u]);
            else load8(static_cast<const float*>(d.g), i, d.n, g[u]);
        }
#pragma unroll
        for (int u = 0; u < kParamChunk / 2048; ++u)
#pragma unroll
            for (int k = 0; k < 8; ++k) sum = fma((double)g[u][k], (double)g[u][k], sum);
    }
    sum = block_sum(sum, red);
    if (threadIdx.x == 0) {
        __hip_atomic_store(&head->part[blockIdx.x], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __threadfence();
        last = atomicInc(&head->norm_ticket, gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    sum = 0.0;
    for (int b = threadIdx.x; b < (int)gridDim.x; b += 256)
        sum += __hip_atomic_load(&head->part[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sum = block_sum(sum, red);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum);
        out[0] = (float)norm;
        out[1] = norm < (double)INFINITY ? (norm > (double)max_norm ? (float)((double)max_norm / norm) : 1.f) : NAN;
    }
}

constexpr int kAdamGroups = 2048;

}  // namespace

hipError_t launch_adamw(int kind, const AdamArgs& a, hipStream_t s) {
    const dim3 g(std::max(1, std::min(a.end - a.first, kAdamGroups))), b(256);
    switch (kind) {
        case 0: hipLaunchKernelGGL((adamw_kernel<0, false, float>), g, b, 0, s, a); break;
        case 1: hipLaunchKernelGGL((adamw_kernel<0, false, uint16_t>), g, b, 0, s, a); break;
        case 2: hipLaunchKernelGGL((adamw_kernel<0, true, float>), g, b, 0, s, a); break;
        case 3: hipLaunchKernelGGL((adamw_kernel<0, true, uint16_t>), g, b, 0, s, a); break;
        case 4: hipLaunchKernelGGL((adamw_kernel<1, false, float>), g, b, 0, s, a); break;
        case 5: hipLaunchKernelGGL((adamw_kernel<1, false, uint16_t>), g, b, 0, s, a); break;
        case 6: hipLaunchKernelGGL((adamw_kernel<1, true, float>), g, b, 0, s, a); break;
        case 7: hipLaunchKernelGGL((adamw_kernel<1, true, uint16_t>), g, b, 0, s, a); break;
        case 8: hipLaunchKernelGGL((adamw_kernel<2, false, float>), g, b, 0, s, a); break;
        case 9: hipLaunchKernelGGL((adamw_kernel<2, false, uint16_t>), g, b, 0, s, a); break;
        case 10: hipLaunchKernelGGL((adamw_kernel<2, true, float>), g, b, 0, s, a); break;
        default: hipLaunchKernelGGL((adamw_kernel<2, true, uint16_t>), g, b, 0, s, a); break;
    }
    return hipGetLastError();
}

hipError_t launch_grad_norm(void* table, size_t descs, size_t map, int chunks, float max_norm, float* out,
                            hipStream_t s) {
    hipLaunchKernelGGL(grad_norm_kernel, dim3(std::max(1, std::min(chunks, kNormGroups))), dim3(256), 0, s,
                       static_cast<unsigned char*>(table), descs, map, chunks, max_norm, out);
    return hipGetLastError();
}

}  // namespace moe
