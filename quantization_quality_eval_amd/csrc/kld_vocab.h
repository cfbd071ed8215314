// Internal interface of the operators at the vocabulary end of a model: beam
// selection over logit rows, reordering of beam states, embedding lookup and
// its gradient. Arguments are validated by the C-ABI host code.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kld_kernels.h"

namespace kldk {

constexpr int kBeamMaxBeams = 64;
constexpr int kBeamMaxSelect = 64;

struct BeamArgs {
    const void* logits;
    int type;             // ElemType
    int64_t vocab;
    int64_t row_stride;   // elements between rows
    int64_t n_items;
    int n_beams;
    int n_select;
    const float* scores;      // [n_items, n_beams]
    const uint8_t* finished;  // [n_items, n_beams] or null
    int eos;                  // -1: none
    float* scores_out;
    int32_t* parents_out;
    int32_t* tokens_out;
    uint8_t* finished_out;
};

int64_t beam_workspace_bytes(int type, int64_t vocab, int64_t n_items, int n_beams, int n_select);
hipError_t launch_beam_select(const BeamArgs& a, void* workspace, hipStream_t stream);

// States of one geometry, reordered in place. Every stride is in bytes; a
// position is position_bytes long and follows the one before it.
struct ReorderArgs {
    void* const* states;  // host array of device pointers
    int n_states;
    int64_t n_items;
    int n_beams;
    const int32_t* parents;
    int64_t beam_stride;
    int64_t n_outer;
    int64_t outer_stride;
    int64_t n_positions;
    int64_t position_bytes;
    const int32_t* lengths;  // device, one per item, or null
};
hipError_t launch_beam_reorder(const ReorderArgs& a, hipStream_t stream);

hipError_t launch_embed(int table_type, int out_type, const void* table, int64_t vocab, int64_t dim,
                        int64_t table_stride, const int32_t* tokens, int64_t n_tokens, double scale, void* out,
                        int64_t out_stride, hipStream_t stream);

struct EmbedGradArgs {
    const void* grad;
    int grad_type;
    int64_t grad_stride;
    const int32_t* tokens;
    int64_t n_tokens;
    int64_t vocab;
    int64_t dim;
    double scale;
    void* out;
    int out_type;
    int64_t out_stride;
    bool accumulate;
};
int64_t embed_grad_workspace_bytes(int64_t vocab, int64_t dim, int64_t n_tokens);
hipError_t launch_embed_grad(const EmbedGradArgs& a, void* workspace, hipStream_t stream);

}  // namespace kldk
