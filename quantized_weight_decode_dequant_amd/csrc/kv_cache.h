// The paged 8-bit cache of keys and values: byte order of a block and the
// argument structs shared by kv_append.hip, kv_attention.hip, kv_tables.hip
// and the C ABI.
//
// A block is what one page (32, 64, 128 or 256 consecutive tokens of a
// request) holds for one KV head: page * D codes, one byte each, with one
// fp32 scale; value = scale * code.  Blocks are stored [pages][Hkv].  Inside
// a block (token t of the page, dimension d) the bytes are ordered so that
// a wave's 128-bit loads are contiguous kilobytes that are already operands
// of the 16x16x32 MFMA:
//   keys    [t/16][d/16][t%16][d%16]: the kilobyte of 16 tokens and 64
//           dimensions gives lane (g = lane >> 4, r = lane & 15) the 16
//           dimensions 16g.. of token r.
//   values  [t/32][d/32][(t%16)/4][d%16][(d/16)%2][(t/16)%2][t%4]: the
//           kilobyte of 32 tokens and 32 dimensions gives lane (g, r) the
//           tokens 4g..4g+3 and 16+4g..16+4g+3 of dimensions r and r + 16,
//           which are the tokens whose scores that lane holds after the
//           product K Q^T, so probabilities never leave their registers.
#pragma once

#include "qg_internal.h"

namespace qg {

constexpr int KV_STEP = 32;          // tokens of one attention step
constexpr int KV_ROWS_MAX = 32;      // query tokens of one request

struct KvAppendArgs {
    uint8_t *k, *v;
    float *k_scales, *v_scales;
    const uint16_t *K, *V;
    const int32_t *slots;
    int64_t k_stride, v_stride;  // elements between tokens
    int64_t slots_end;           // pages * page
    int M, Hkv, D, page, chunk;
};

struct KvAttnArgs {
    const uint8_t *k, *v;
    const float *k_scales, *v_scales;
    const uint16_t *q;
    const int32_t *q_start, *lens, *table;
    const uint32_t *tree;
    void *out;
    float *part;     // [part_slots][part_rows][D]: a segment's unnormalised sums
    float *part_ml;  // [part_slots][part_rows][2]: its running maximum (base 2) and sum
    int64_t q_stride, out_stride;  // elements between tokens
    int64_t pages;
    int R, M, Hq, Hkv, G, page, max_blocks, max_q, max_len, window;
    int groups, slots, min_run, part_rows, part_slots;  // of KvAttnPlan
    int32_t *head;       // run length, then where each request's work starts
    bool whole, aligned;
    float scale;     // softmax scale * log2(e)
    bool out_f32;
};

struct KvTablesArgs {
    int32_t *lens, *table, *free_pages, *free_count;
    const int32_t *keep, *add;
    int32_t *q_start, *slots, *positions, *status;
    int64_t pages;
    int R, page, page_bits, max_blocks, max_tokens;
};

hipError_t launch_kv_append(const KvAppendArgs &a, bool e4m3, hipStream_t s);
hipError_t launch_kv_attention(const KvAttnArgs &a, int D, bool e4m3, hipStream_t s);
hipError_t launch_kv_tables(const KvTablesArgs &a, hipStream_t s);
// How an attention call is cut; false where its work does not fit 31 bits.
struct KvAttnPlan {
    int groups;          // row groups of a request of max_q tokens
    int slots;           // workgroups that share the work
    int min_run;         // steps one of them takes at least
    int part_rows;       // rows of a segment
    int64_t part_slots;  // places for segments
    int64_t head_bytes;  // in front of them
    bool aligned;        // a cut falls on the start of every (request, head, row group)
    bool whole;          // nothing is cut: a workgroup for each (request, head, row group)
};
bool kv_attention_plan(int64_t R, int64_t Hkv, int64_t G, int64_t D, int64_t max_q, int64_t seen, KvAttnPlan *p);

constexpr int KV_R_MAX = 4096;       // requests of a call

}  // namespace qg
