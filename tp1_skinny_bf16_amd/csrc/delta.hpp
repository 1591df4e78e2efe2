// delta.hpp -- the gated delta rule: the launch interface of its recurrent
// (delta_step.hip) and chunked (delta_chunk.hip) kernels, and what a token's
// gate is.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/tp1_proj.h"

namespace tp1 {

constexpr int kHead = PROJ_DELTA_HEAD;  // key and value size of a head

struct DeltaArgs {
    const uint16_t *q, *k, *v, *f, *b;  // BF16 rows
    long ldq, ldk, ldv, ldf, ldb;       // row strides in elements
    const float *a_log, *dt_bias;
    float *state;                       // [n_slots][H][key][value]
    uint16_t *out;
    long ldo;
    float scale;                        // of q
    int l2norm;
    int H, rep;                         // value heads, and how many share a key head
    int n_slots;
};

// Which rows and which state a sequence has: from a device table of
// {first row, rows, slot} (slots checked on the host, no two alike), or
// request i has rows [i * tokens, (i + 1) * tokens) and slots[i].
struct DeltaSeqs {
    const int *table;
    const int *slots;
    int tokens;
    int n;
};

// The chunked form.
constexpr int kDeltaChunk = 64;             // tokens a chunk
constexpr int kDeltaItemBytes = 107520;     // workspace of a chunk and head
constexpr int kDeltaLds = 77824;            // LDS of a workgroup: two a compute unit

// A segment of the chunks: which to prepare, and which sequences to carry on.
struct DeltaSegment {
    const int *chunk_table;  // {first row, rows} a chunk, by place in the workspace
    const int *seq_table;    // {first row, rows, slot, first chunk} a sequence
    char *ws;
    int chunks, seqs;
    int longest;             // most chunks of one sequence here
};

hipError_t launch_delta_steps(const DeltaArgs &a, const DeltaSeqs &s, bool head_gate, int cus,
                              hipStream_t st);

// The scan of one segment and the preparation of the next (either may be
// empty) in one launch.
hipError_t launch_delta_chunks(const DeltaArgs &a, const DeltaSegment &scan,
                               const DeltaSegment &prep, bool head_gate, int cus,
                               hipStream_t st);
// Allow the chunk kernels their LDS on the current device.
hipError_t allow_delta_lds();

#ifdef __HIPCC__
// ln of a token's decay: -exp(A_log) * softplus(f + dt_bias).
__device__ __forceinline__ float log_decay(float rate, float f, float bias) {
    const float z = f + bias;
    return -rate * (fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))));
}
__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }
// Added to a squared length before its root.
constexpr float kUnitEps = 1e-6f;
#endif

}  // namespace tp1
