// Internal declarations of the operators of include/kda_beam.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_beam.h"
#include "kda_internal.cuh"

namespace kda {

struct BeamSelectIO {
    int groups, beams, vocab;
    const void* logits;
    int bf16;
    long long row_stride;
    const float* scores;
    const uint8_t* done;   // may be null
    int end_token, num, keep;
    float* out_scores;
    int* out_tokens;
    int* out_rows;
    void* workspace;
};

struct BeamReorderIO {
    int B;
    const int* rows;
    const uint8_t* src[2];   // S and the conv windows
    uint8_t* dst[2];
    long long bytes[2];      // of one sequence
    bool in_place;
};

size_t beam_select_workspace_bytes(int groups, int beams, int vocab, int num, const DeviceInfo& dev);
cudaError_t launch_beam_select(const BeamSelectIO& io, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_beam_reorder(const BeamReorderIO& io, const DeviceInfo& dev, int* err_word, cudaStream_t stream);

}  // namespace kda
