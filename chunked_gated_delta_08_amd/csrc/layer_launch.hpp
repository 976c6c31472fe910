// layer_launch.hpp -- host-side launchers of the layer operators (include/gdn_layer.h; internal).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace layer {

// Dropout (gdn_dropout): the host's part of the mask.
struct Drop {
    uint64_t seed, offset;
    const uint64_t* rng;   // device seed and offset, or NULL
    uint32_t drop;         // of 65536, how many values drop an element
    float mul;             // 65536 / (65536 - drop)
};
hipError_t launch_dropout(int dtype, const void* x, void* y, int64_t rows, int64_t D, const Drop& d, hipStream_t s);

// Both norms.  E: dtype (gdr_dtype), R: type of the residual stream.
struct NormArgs {
    long rows;
    int D;
    float eps;
    int dtype, res_dtype;
    int act;                      // gdn_act
    const void* x; const void* z; // z NULL: no gate
    const float* w; const float* scale;
    const void* res; const void* dy; const void* dres;
    void* y; void* res_out;       // forward
    void* dx; void* dz; void* dres_out;
    float* dw; float* dscale;
    float* part; float* part_s;   // backward: the workgroups' column sums for dw and dscale, `pitch` floats apart
    int pitch;
    bool dropped; Drop drop;      // add norm: whether the branch x is dropped out, and how
};

// Floats of `part` that either backward may use.
size_t norm_part_floats(long rows, int D);
hipError_t launch_gated_norm_fwd(const NormArgs& a, hipStream_t s);
hipError_t launch_gated_norm_bwd(const NormArgs& a, hipStream_t s);
hipError_t launch_add_norm_fwd(const NormArgs& a, hipStream_t s);
hipError_t launch_add_norm_bwd(const NormArgs& a, hipStream_t s);

// Gated linear recurrence.
struct GlrArgs {
    long ntok;                 // tokens of the flattened axis
    int nseq, T;               // sequences; dense length
    int D, dtype;
    int polls;                 // tries before a workgroup takes up what it waits for
    const int32_t* cu;         // device cu_seqlens or NULL
    const void* x; const float* g; const float* h0;
    void* h; float* ht; float* states;            // forward outputs; backward reads states
    const void* dh; const float* dht; void* dx; float* dg; float* dh0;
    void* ws;
};
size_t glr_ws_bytes(const GlrArgs& a);
long glr_threads(const GlrArgs& a);   // of the larger launch
hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t s);
hipError_t launch_glr_bwd(const GlrArgs& a, hipStream_t s);

struct StepArgs {
    int N, HK, HV, K, D;       // gdr_step: K = V; glr_step: D channels
    long nslots;
    float scale;
    int dtype;
    const void* q; const void* k; const void* v; const float* g; const void* beta;
    const int32_t* slots;
    float* state;
    void* o;
};
hipError_t launch_glr_step(const StepArgs& a, hipStream_t s);
hipError_t launch_gdr_step(const StepArgs& a, hipStream_t s);

}  // namespace layer
