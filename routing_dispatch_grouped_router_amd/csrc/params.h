// The table of an optimizer's tensors as the kernels read it: written on the
// host by moe_param_table, copied to the device by the caller.
//
//   ParamHead | ParamDesc [tensors with elements] | uint32_t [chunks]
//
// A chunk is kParamChunk consecutive elements of one tensor (the last of a
// tensor may be shorter); chunk c belongs to tensor descs[map[c]].  Chunks are
// ordered by kind, so that a launch takes those of one kind.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kParamBlock = 128;       // elements of an 8-bit moment that share a scale
constexpr int kParamChunk = 2048;      // eight elements a thread
constexpr int kNormGroups = 1024;      // most workgroups of the norm, and partial sums

// Kinds: 4 * (weights: 0 float32, 1 bfloat16 with a float32 master, 2 bfloat16 alone)
// + 2 * (8-bit moments) + (bfloat16 gradients); kKindNorm: no weight, for the norm only.
constexpr int kKinds = 12;
constexpr int kKindNorm = kKinds;

struct ParamDesc {
    void* w;
    const void* g;
    float* master;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    uint64_t n;
    float lr_scale, decay;
    uint32_t index;        // the tensor's place in the caller's list
    uint32_t first;        // its first chunk
    int32_t g_bf16;
    int32_t pad;
};
static_assert(sizeof(ParamDesc) == 88, "read by the kernels as it is written here");

// Counters that find the last workgroup of a launch, zero between launches.  One
// address takes an atomic of the whole card every 30 to 70 ns (1024 workgroups: 65
// us), so workgroups count in 32 groups, each on a line of its own, and the
// groups' last ones once more.
struct Tickets {
    uint32_t group[32][16];
    uint32_t all[16];
};

struct ParamHead {
    Tickets norm, step;
    double part[kNormGroups];
};

struct AdamArgs {
    unsigned char* table;
    size_t descs, map;     // offsets in the table
    int first, end;        // chunks of this launch
    const float* lr;       // [1]
    const float* clip;     // [2], the second used; NULL: 1
    int32_t* step;         // [2]: steps taken; not used
    bool nt;               // whether the tensors are streamed past the caches
    int count;             // whether this launch, the step's last, counts it
    uint32_t seed;
    double beta1, beta2;
    float eps;
};

}  // namespace moe
