// Arguments and workspace of the sampling kernels (sample.hip), filled by the
// C ABI.
#pragma once

#include "qg_internal.h"

namespace qg {

constexpr int64_t SAMPLE_V_MAX = int64_t(1) << 20;
constexpr int SAMPLE_THREADS = 256;
constexpr int SAMPLE_PER_THREAD = 16;
constexpr int SAMPLE_CHUNK = SAMPLE_THREADS * SAMPLE_PER_THREAD;  // tokens of one workgroup
constexpr int SAMPLE_BINS = 2048;
constexpr int SAMPLE_LIST = 8192;  // a row's undecided tokens that are kept as a list
constexpr int SAMPLE_SUBS = SAMPLE_THREADS / 64;  // parts of a chunk, a wave's 1024 tokens each
static_assert(SAMPLE_V_MAX / SAMPLE_CHUNK <= SAMPLE_THREADS, "a row's chunks are one for each thread");

// What a row's kernels leave for each other.
struct SampleRow {
    int done;                   // the token is written already
    int full;                   // bins below are kept whole
    int p_lo, p_hi;             // bins among which top-p's border lies (p_lo > p_hi: none)
    int k_bin;                  // the bin of top-k's border (-1: none)
    unsigned k_left;            // tokens of k_bin that top-k keeps
    unsigned listed;            // undecided tokens (those in the border's bins)
    float top;                  // the row's largest logit
    unsigned long long p_mass;  // mass of the bins below p_lo
    unsigned long long k_mass;  // mass of the bins below k_bin
    unsigned long long mass;    // of all bins
};

struct SampleArgs {
    const void *logits;
    int64_t stride;  // elements between rows
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *tokens;
    float *logprobs;
    // workspace, by row
    SampleRow *rows;             // [M]
    unsigned long long *masses;  // [M][SAMPLE_BINS]
    unsigned *counts;            // [M][SAMPLE_BINS]
    unsigned long long *kept;    // [M][chunks][SAMPLE_SUBS]: mass that is kept for sure
    float *tops;                 // [M][chunks][SAMPLE_SUBS]: largest logit
    int32_t *top_at;             // [M][chunks][SAMPLE_SUBS]: the first token that has it (-1: all are NaN)
    u32x2_t *lists;              // [M][SAMPLE_LIST]: (key, token) of undecided tokens
    int M, V, chunks;
    bool few;  // workgroups: they read ahead of a row's settings, and find its borders each
};

hipError_t launch_sample(const SampleArgs &a, bool x_f32, hipStream_t s);

}  // namespace qg
