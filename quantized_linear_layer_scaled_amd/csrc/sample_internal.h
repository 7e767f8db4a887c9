// Internal declarations of the sampler.  Not part of the public interface
// (see include/qll.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qll {

constexpr int kSampleMaxVocab = 1 << 20;

struct SampleArgs {
    const void* logits;  // [B] rows of V values, ld apart
    int64_t ld;
    int bf16;
    const float* u;            // [B]
    const float* temperature;  // [B] or null, and so on
    const int* top_k;
    const float* top_p;
    const float* min_p;
    int* tokens;   // [B]
    float* probs;  // [B] or null
    int B, V;
    int ebits;  // fixed-point bits of a bin's complement (see sample.hip)
    int parts;  // workgroups of a row
    void* ws;   // B * parts * sample_part_bytes() where parts > 1
};
constexpr int kSamplePartList = 1024;
int sample_parts(int64_t B, int64_t V);
int64_t sample_part_bytes();
hipError_t launch_sample(const SampleArgs& a, hipStream_t stream);

}  // namespace qll
