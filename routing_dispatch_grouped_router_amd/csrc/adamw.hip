// The end of a training step over many tensors at once, for gfx950: the norm of
// all gradients, and the AdamW step.
//
//   norm = sqrt(sum over all tensors of g^2),  factor = max_norm / norm if norm > max_norm, else 1
//   t = steps taken + 1,  g' = factor g,
//   m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2,
//   w = w - lr (m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps) + decay w).
//
// One launch for all tensors of a kind: a table in device memory says where they
// are, a workgroup takes chunks of 2048 elements, eight consecutive ones a
// thread, so that every stream moves in 16-byte pieces.  The wave that holds a
// tensor's end goes element by element; nothing outside a tensor is touched.
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
// A positive root has a code of 1 at least.  Both moments' smallest codes are
// 1/229376 of their block's largest values; a root cut to 0 beside an m that has
// a code would leave the next step m over little more than eps (blocks whose
// elements differ by 10^5 and more: steps of 400 to 700 lr, 2.2 with the code).
// The steps of an element that far below its block's largest are too small
// instead, as its root is held too large.
// A root that is right on average has a square too large by the rounding's
// variance.  A step leaves r close to the code it came from, a part f of the way to
// the next that is in proportion to 1 - b2, and the variance f (1 - f) with it: v
// is larger by 3 to 4 % on average whatever b2 is (gradients of a normal
// distribution, b2 from 0.95 to 0.999), its root by half of that.
//
// HBM bounds it: an element's 30 bytes (bf16 weight, float32 master, moments and
// gradient), 28 (float32) or 12 (bf16 alone, 8-bit moments) are read and
// written once.  50 M elements (three 8 x 2048 x 1024 tensors and small ones):
// norm 38 us, 5.2 TB/s; step of bf16 with masters 287 us, 5.3 TB/s; with 8-bit
// moments and no master 133 us, 4.6 TB/s, passes back to back (launches under a
// trace, with gaps between them, 289 and 156; a 2 GiB copy runs at 4.9 TB/s on the
// same card).
#include <algorithm>

#include "moe_device.h"
#include "moe_internal.h"
#include "params.h"

namespace moe {

namespace {

// ----------------------------------------------------------------------------- eight elements of a stream

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// The tensors' addresses come from memory: said to be global here, so that they
// are not accessed as what might be LDS too.
template <typename T>
using Global = __attribute__((address_space(1))) T;

template <typename T, bool NT>
__device__ __forceinline__ T get(const void* p) {
    const Global<T>* q = (const Global<T>*)p;
    return NT ? __builtin_nontemporal_load(q) : *q;
}
template <typename T, bool NT>
__device__ __forceinline__ void put(void* p, T v) {
    Global<T>* q = (Global<T>*)p;
    if (NT) __builtin_nontemporal_store(v, q);
    else *q = v;
}

// Elements [i, i + 8) of p as float32; unless FULL those below n, and zero from n on.
template <bool NT, bool FULL>
__device__ __forceinline__ void load8(const float* p, uint64_t i, uint64_t n, float (&v)[8]) {
    if (FULL) {
        const u32x4 a = get<u32x4, NT>(p + i), b = get<u32x4, NT>(p + i + 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = __uint_as_float(a[k]);
            v[4 + k] = __uint_as_float(b[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = i + k < n ? get<float, false>(p + i + k) : 0.f;
    }
}
template <bool NT, bool FULL>
__device__ __forceinline__ void load8(const uint16_t* p, uint64_t i, uint64_t n, float (&v)[8]) {
    if (FULL) {
        unpack16<true>(get<u32x4, NT>(p + i), v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = i + k < n ? bf16_to_f32(get<uint16_t, false>(p + i + k)) : 0.f;
    }
}
template <bool NT, bool FULL>
__device__ __forceinline__ void store8(float* p, uint64_t i, uint64_t n, const float (&v)[8]) {
    if (FULL) {
        u32x4 a, b;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            a[k] = __float_as_uint(v[k]);
            b[k] = __float_as_uint(v[4 + k]);
        }
        put<u32x4, NT>(p + i, a);
        put<u32x4, NT>(p + i + 4, b);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + k < n) put<float, false>(p + i + k, v[k]);
    }
}
template <bool NT, bool FULL>
__device__ __forceinline__ void store8(uint16_t* p, uint64_t i, uint64_t n, const float (&v)[8]) {
    if (FULL) {
        put<u32x4, NT>(p + i, pack16<true>(v));
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + k < n) put<uint16_t, false>(p + i + k, f32_to_bf16(v[k]));
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

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Eight codes (zero from n on).
template <bool NT, bool FULL>
__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, uint64_t i, uint64_t n) {
    u32x2 w = {0u, 0u};
    if (FULL) {
        w = get<u32x2, NT>(p + i);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + k < n) w[k / 4] |= (uint32_t)get<uint8_t, false>(p + i + k) << (8 * (k % 4));
    }
    return w;
}
__device__ __forceinline__ void decode(u32x2 w, float scale, float (&v)[8]) {
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
// a block call it together.  Random bits of value k: the low (HIGH: high) half of
// h[k].  A value's exponent and fraction as E4M3 has them stand above 20 further
// bits once it is times 2^-120: 20 random bits (16 and a half) are added there
// and the sum cut.  Infinite and NaN values get the NaN code and do not count for
// the scale; a block below 2^-100 is zero.  SIGNED false, roots: no value is below
// 0 (the smallest above it is 2^-75), and a code is 0 only for 0.
template <bool NT, bool FULL, bool HIGH, bool SIGNED>
__device__ __forceinline__ void store_codes(uint8_t* p, float* scales, uint64_t i, uint64_t n, const float (&v)[8],
                                            const uint32_t (&h)[8]) {
    uint32_t top = 0u;   // of the magnitudes' bits, which order as the magnitudes do
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(v[k]) & 0x7FFFFFFFu);
    top = group_reduce<16>(top, MaxU32());
    const bool finite = top < 0x7F800000u;
    if (!finite) {
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(v[k]) < INFINITY ? fabsf(v[k]) : 0.f);
        top = group_reduce<16>(__float_as_uint(amax), MaxU32());   // the 16 lanes of a block are here or not together
    }
    float amax = __uint_as_float(top);
    if (amax < 0x1p-100f) amax = 0.f;
    // products with rounded reciprocals, as the definition has them (quotients would be another float32 in half of all
    // blocks, and the step of 50 M elements take 135 us instead of 132)
    if (i % kParamBlock == 0 && (FULL || i < n)) put<float, false>(scales + i / kParamBlock, amax * (1.f / 448.f));
    const float inv = amax > 0.f ? 1.f / amax * 448.f : 0.f;
    u32x2 w = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t u = __float_as_uint(fminf(fabsf(v[k]) * inv, 448.f) * 0x1p-120f);
        const uint32_t r = HIGH ? (h[k] >> 12) & 0xFFFF0u : (h[k] << 4) & 0xFFFF0u;
        uint32_t c = min((u + (r | 8u)) >> 20, 0x7Eu);
        if (SIGNED) c |= (__float_as_uint(v[k]) >> 24) & 0x80u;
        else c = max(c, min(__float_as_uint(v[k]), 1u));
        w[k / 4] |= c << (8 * (k % 4));
    }
    if (!finite) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (!(fabsf(v[k]) < INFINITY)) w[k / 4] |= 0x7Fu << (8 * (k % 4));
    }
    if (FULL) {
        put<u32x2, NT>(p + i, w);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + k < n) put<uint8_t, false>(p + i + k, (uint8_t)(w[k / 4] >> (8 * (k % 4))));
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

// The square root, of values that may be denormal or 0: Newton's step for the root from the reciprocal root's
// instruction (1 step off), which leaves a value in a million not the nearest.
__device__ __forceinline__ float root(float v) {
#pragma clang fp contract(off)
    const bool tiny = v < 0x1p-60f;
    const float x = v * (tiny ? 0x1p64f : 1.f), y = __builtin_amdgcn_rsqf(fmaxf(x, 0x1p-90f)), r = x * y;
    return x < INFINITY ? fmaf(fmaf(-r, r, x), 0.5f * y, r) * (tiny ? 0x1p-32f : 1.f) : x;
}

struct StepScalars {
    float factor, lr, c1, c2_root, b1, g1, b2, g2, eps;   // c1 = 1 / (1 - b1^t), c2_root = 1 / sqrt(1 - b2^t)
    uint32_t key;
};

// One chunk, from element `base` on, FULL or the last of its tensor.  W: weights float32 (0), bfloat16 with a master (1),
// bfloat16 alone (2).
template <int W, bool S8, typename G, bool NT, bool FULL>
__device__ __forceinline__ void adamw_chunk(const ParamDesc& d, uint64_t base, const StepScalars& s, uint32_t key) {
#pragma clang fp contract(off)
    const uint64_t i = base + 8 * threadIdx.x;
    float g[8], w[8], m[8], v[8], r[8];
    load8<NT, FULL>(static_cast<const G*>(d.g), i, d.n, g);
    if (W == 0) load8<NT, FULL>(static_cast<const float*>(d.w), i, d.n, w);
    else if (W == 1) load8<NT, FULL>(d.master, i, d.n, w);
    else load8<NT, FULL>(static_cast<const uint16_t*>(d.w), i, d.n, w);
    if (S8) {
        const u32x2 mc = load_codes<NT, FULL>(static_cast<const uint8_t*>(d.m), i, d.n);
        const u32x2 rc = load_codes<NT, FULL>(static_cast<const uint8_t*>(d.v), i, d.n);
        const float ms = FULL || i < d.n ? get<float, false>(d.m_scale + i / kParamBlock) : 0.f;
        const float rs = FULL || i < d.n ? get<float, false>(d.v_scale + i / kParamBlock) : 0.f;
        decode(mc, ms, m);
        decode(rc, rs, r);
    } else {
        load8<NT, FULL>(static_cast<const float*>(d.m), i, d.n, m);
        load8<NT, FULL>(static_cast<const float*>(d.v), i, d.n, v);
    }
    const float lr = s.lr * d.lr_scale;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        // each operation of the formula rounded, as anyone's would be: a code hangs on m's and r's last bits
        const float gk = g[k] * s.factor;
        m[k] = s.b1 * m[k] + s.g1 * gk;
        v[k] = s.b2 * (S8 ? r[k] * r[k] : v[k]) + s.g2 * gk * gk;
        r[k] = root(v[k]);
        const float step = m[k] * s.c1 * __builtin_amdgcn_rcpf(fmaf(r[k], s.c2_root, s.eps));
        w[k] = fmaf(-lr, fmaf(d.decay, w[k], step), w[k]);
    }
    uint32_t h[8];
    if (S8 || W == 2) {
        const uint32_t first = mix(key ^ (uint32_t)(i / kParamBlock)) + (uint32_t)(i % kParamBlock) * 0x9E3779B9u;
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] = mix(first + k * 0x9E3779B9u);
    }
    if (S8) {
        store_codes<NT, FULL, false, true>(static_cast<uint8_t*>(d.m), d.m_scale, i, d.n, m, h);
        store_codes<NT, FULL, true, false>(static_cast<uint8_t*>(d.v), d.v_scale, i, d.n, r, h);
    } else {
        store8<NT, FULL>(static_cast<float*>(d.m), i, d.n, m);
        store8<NT, FULL>(static_cast<float*>(d.v), i, d.n, v);
    }
    if (W == 0) {
        store8<NT, FULL>(static_cast<float*>(d.w), i, d.n, w);
        return;
    }
    if (W == 1) {
        store8<NT, FULL>(d.master, i, d.n, w);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t up = __float_as_uint(w[k]) + (mix(h[k] + 0x7F4A7C15u) & 0xFFFFu);
            if (fabsf(w[k]) < INFINITY) w[k] = __uint_as_float(up & 0xFFFF0000u);
        }
    }
    store8<NT, FULL>(static_cast<uint16_t*>(d.w), i, d.n, w);
}

// The tensor that a workgroup's chunk belongs to, read again where it changes.
struct Tensor {
    ParamDesc d;
    int end = 0;   // the first chunk past it
    __device__ __forceinline__ bool at(const ParamDesc* descs, const uint32_t* map, int c) {
        if (c < end) return false;
        d = descs[map[c]];
        end = (int)(d.first + (d.n + kParamChunk - 1) / kParamChunk);
        return true;
    }
    __device__ __forceinline__ uint64_t base(int c) const { return (uint64_t)(c - (int)d.first) * kParamChunk; }
};

// Whether this workgroup (its one thread that asks) is the last to ask.
__device__ __forceinline__ bool last_to_ask(Tickets& t) {
    const uint32_t g = blockIdx.x % 32, members = (gridDim.x - g + 31) / 32, groups = min(gridDim.x, 32u);
    return atomicInc(&t.group[g][0], members - 1) == members - 1 && atomicInc(&t.all[0], groups - 1) == groups - 1;
}

template <int W, bool S8, typename G, bool NT>
__global__ __launch_bounds__(256) void adamw_kernel(AdamArgs a) {
    const ParamDesc* descs = reinterpret_cast<const ParamDesc*>(a.table + a.descs);
    const uint32_t* map = reinterpret_cast<const uint32_t*>(a.table + a.map);
    Tensor tensor;
    int c = a.first + blockIdx.x;
    if (c < a.end) tensor.at(descs, map, c);   // requested before what the step needs is worked out
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
        uint32_t key = mix(s.key + tensor.d.index);
        for (; c < a.end; c += gridDim.x) {
            if (tensor.at(descs, map, c)) key = mix(s.key + tensor.d.index);
            const uint64_t base = tensor.base(c);
            if (!S8) __syncthreads();   // waves side by side in each stream: 293 us instead of 302 (below)
            // the last chunk of a tensor: whole waves as in the others, element by element where its end is
            if (base + kParamChunk <= tensor.d.n || base + 512 * (uniform(threadIdx.x >> 6) + 1) <= tensor.d.n)
                adamw_chunk<W, S8, G, NT, true>(tensor.d, base, s, key);
            else
                adamw_chunk<W, S8, G, NT, false>(tensor.d, base, s, key);
        }
    }
    if (!a.count) return;
    __syncthreads();   // every wave has read the count
    // the last workgroup to come here counts the step: every other one has read the count
    if (threadIdx.x == 0 && last_to_ask(reinterpret_cast<ParamHead*>(a.table)->step) && finite) a.step[0] = taken + 1;
}

// ----------------------------------------------------------------------------- the norm

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return ((red[0] + red[1]) + red[2]) + red[3];
}

// The squares of the chunks of p at e0, e0 + by, ... below e1, on top of sum.
template <typename G, bool NT>
__device__ __forceinline__ double squares(const G* p, uint64_t e0, uint64_t e1, uint64_t by, uint64_t n, double sum) {
    constexpr int kB = 4;   // chunks in flight
    for (uint64_t e = e0; e < e1; e += kB * by) {
        float g[kB][8];
#pragma unroll
        for (int u = 0; u < kB; ++u) {
            const uint64_t c = e + u * by;
            if (c >= e1) continue;
            if (c + 512 * (uniform(threadIdx.x >> 6) + 1) <= n) load8<NT, true>(p, c + 8 * threadIdx.x, n, g[u]);
            else load8<NT, false>(p, c + 8 * threadIdx.x, n, g[u]);
        }
#pragma unroll
        for (int u = 0; u < kB; ++u)
            if (e + u * by < e1) {
#pragma unroll
                for (int k = 0; k < 8; ++k) sum = fma((double)g[u][k], (double)g[u][k], sum);
            }
    }
    return sum;
}

// Squares summed in float64 (no float32 value's square leaves its range), a
// workgroup's chunks in order, the workgroups' sums in order by the last of them.
template <bool NT>
__global__ __launch_bounds__(256) void grad_norm_kernel(unsigned char* table, size_t descs_at, size_t map_at,
                                                        int chunks, float max_norm, float* __restrict__ out) {
    __shared__ double red[4];
    __shared__ bool last;
    ParamHead* head = reinterpret_cast<ParamHead*>(table);
    const ParamDesc* descs = reinterpret_cast<const ParamDesc*>(table + descs_at);
    const uint32_t* map = reinterpret_cast<const uint32_t*>(table + map_at);
    double sum = 0.0;
    Tensor t;
    for (int c = blockIdx.x; c < chunks; c += (t.end - c + gridDim.x - 1) / gridDim.x * gridDim.x) {
        t.at(descs, map, c);
        const uint64_t by = (uint64_t)gridDim.x * kParamChunk;
        sum = t.d.g_bf16 ? squares<uint16_t, NT>(static_cast<const uint16_t*>(t.d.g), t.base(c), t.d.n, by, t.d.n, sum)
                         : squares<float, NT>(static_cast<const float*>(t.d.g), t.base(c), t.d.n, by, t.d.n, sum);
    }
    sum = block_sum(sum, red);
    if (threadIdx.x == 0) {
        // the sum is written through to where every XCD sees it, and has arrived, before this workgroup asks: no
        // fence, which would write back and invalidate an L2 for each workgroup
        __hip_atomic_store(&head->part[blockIdx.x], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        last = last_to_ask(head->norm);
    }
    __syncthreads();
    if (!last) return;
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

// Workgroups.  32-bit moments: one or two a compute unit, through the caches:
// six to eight streams are DRAM's to keep apart, and more of them at once scatter
// its accesses (50 M elements, bf16 with master: 256 workgroups 287 us, 5.3 TB/s;
// 512 293, 1024 and 2048 300, past the caches 295 to 345, 384 and 640 workgroups
// 340).  Smaller sets gain from the second: 0.8 M elements 9.3 and 8.4 us with 256
// and 512; with masters 17 M 95.3 and 86.4, 21 M 120.4 and 118.0, 26 M 153.4 and
// 155.5; float32 17 M 72.2 and 71.3, 21 M 109.3 and 103.6, 26 M 140.5 and 141.8: 256
// from 23 M on.  8-bit moments: 2048, past the caches: the arithmetic (300 cycles
// an element of a wave's 64) needs the waves (without the roots' least code 131 us,
// 1024 workgroups 134, 512 161, through the caches 137; with it 133).
template <int W, bool S8, typename G>
void launch_kind(const AdamArgs& a, hipStream_t s) {
    const int chunks = a.end - a.first, most = S8 ? 2048 : (chunks >= 11264 ? 256 : 512);
    const dim3 g(std::max(1, std::min(chunks, most))), b(256);
    if (S8 && a.nt) hipLaunchKernelGGL((adamw_kernel<W, S8, G, S8>), g, b, 0, s, a);
    else hipLaunchKernelGGL((adamw_kernel<W, S8, G, false>), g, b, 0, s, a);
}

}  // namespace

hipError_t launch_adamw(int kind, const AdamArgs& a, hipStream_t s) {
    switch (kind) {
        case 0: launch_kind<0, false, float>(a, s); break;
        case 1: launch_kind<0, false, uint16_t>(a, s); break;
        case 2: launch_kind<0, true, float>(a, s); break;
        case 3: launch_kind<0, true, uint16_t>(a, s); break;
        case 4: launch_kind<1, false, float>(a, s); break;
        case 5: launch_kind<1, false, uint16_t>(a, s); break;
        case 6: launch_kind<1, true, float>(a, s); break;
        case 7: launch_kind<1, true, uint16_t>(a, s); break;
        case 8: launch_kind<2, false, float>(a, s); break;
        case 9: launch_kind<2, false, uint16_t>(a, s); break;
        case 10: launch_kind<2, true, float>(a, s); break;
        default: launch_kind<2, true, uint16_t>(a, s); break;
    }
    return hipGetLastError();
}

hipError_t launch_grad_norm(void* table, size_t descs, size_t map, int chunks, float max_norm, float* out,
                            hipStream_t s) {
    const dim3 g(std::max(1, std::min(chunks, kNormGroups))), b(256);
    unsigned char* t = static_cast<unsigned char*>(table);
    if (past_caches((size_t)chunks * kParamChunk * 4))
        hipLaunchKernelGGL(grad_norm_kernel<true>, g, b, 0, s, t, descs, map, chunks, max_norm, out);
    else
        hipLaunchKernelGGL(grad_norm_kernel<false>, g, b, 0, s, t, descs, map, chunks, max_norm, out);
    return hipGetLastError();
}

}  // namespace moe
