// Host-side interface between the row operators' C ABI (rows_api.cu) and
// their kernels (route.cu, expert.cu, embedding.cu, beam.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "launch.h"

namespace gbs {

enum RowType : int { ROW_F32 = 0, ROW_F16 = 1, ROW_BF16 = 2 };
constexpr int row_bytes(int type) { return type == ROW_F32 ? 4 : 2; }

// Starts a call: clears the launch count and records the first timing event
// (api.cu).  Returns the calling thread's launch counter.
int *call_begin(cudaStream_t stream);

int device_sm_count();

// A matrix of rows: row i starts at base + i * stride values.
struct Rows {
    void *base;
    size_t stride;
    int type;
};

// Largest number of values, a power of two, that one access may cover: every
// row starts on a multiple of it (at most 16 bytes), and it divides the row.
inline int pack_values(const Rows *rows, int count, size_t row_len) {
    int n = 8;
    for (int i = 0; i < count; ++i) {
        const size_t b = (size_t)row_bytes(rows[i].type);
        while (n > 1 && ((reinterpret_cast<uintptr_t>(rows[i].base) % (n * b < 16 ? n * b : 16)) != 0 ||
                         (rows[i].stride * b) % (n * b < 16 ? n * b : 16) != 0 || row_len % (size_t)n != 0))
            n /= 2;
    }
    return n;
}

// Whether every row starts at and consists of whole units of 16 bytes.
inline bool whole_packs(const Rows *rows, int count, size_t row_len) {
    for (int i = 0; i < count; ++i) {
        const size_t b = (size_t)row_bytes(rows[i].type);
        if ((reinterpret_cast<uintptr_t>(rows[i].base) | rows[i].stride * b | row_len * b) % 16 != 0) return false;
    }
    return true;
}

// Of `count` ids from `first` on, those that 64 bits have: a range that would
// end past 2^63 - 1 ends there.
inline uint64_t ids_from(int64_t first, uint64_t count) {
    const uint64_t last = (uint64_t)INT64_MAX - (uint64_t)first;
    return count != 0 && count - 1 > last ? last + 1 : count;
}

// The slots (t, k) of one call, grouped by expert.
struct ExpertJob {
    const void *ids;
    int id_bytes;
    size_t num_tokens;
    uint32_t top_k;
    uint32_t num_experts;
    int64_t first_expert;
    uint32_t row_align;
    size_t num_rows;
    int32_t *slot_of_row, *row_of_slot, *offsets, *counts;
    Header *hdr;
    uint32_t *tile_counts;  // work buffer: [tiles][num_experts], see expert_temp_bytes
    Rows x, rows;           // x.base == nullptr: no rows are moved
    size_t row_len;
};
size_t expert_temp_bytes(size_t num_tokens, size_t top_k, size_t num_experts);
cudaError_t launch_expert_dispatch(const ExpertJob &job, cudaStream_t stream, int *launches);

struct ExpertMoveJob {
    const int32_t *slot_of_row, *row_of_slot;
    size_t num_tokens, num_rows, row_len;
    uint32_t top_k;
    int weight_type;
    const void *weights;  // nullptr: ones
    Rows x;               // [num_tokens]: the tokens' rows (gather: in; combine: out; combine_grad: d_out)
    Rows rows;            // [num_rows]: the experts' rows
    Rows d_rows;          // combine_grad only
    void *d_weights;      // combine_grad only; nullptr: not computed
};
cudaError_t launch_expert_gather(const ExpertMoveJob &job, cudaStream_t stream, int *launches);
cudaError_t launch_expert_combine(const ExpertMoveJob &job, cudaStream_t stream, int *launches);
cudaError_t launch_expert_combine_grad(const ExpertMoveJob &job, cudaStream_t stream, int *launches);

// A router's choice, or its gradient (route.cu).
struct RouteJob {
    Rows logits;  // [num_tokens][num_experts]
    size_t num_tokens;
    uint32_t num_experts, top_k;
    bool sigmoid, renormalise;
    float scale;
    const float *bias;  // route only; nullptr: none
    uint32_t num_groups, top_groups, group_top;  // route only
    void *ids;
    int id_bytes;
    void *weights;  // grad: their gradient
    int weight_type;
    Rows d_logits;  // grad only
};
cudaError_t launch_route(const RouteJob &job, cudaStream_t stream, int *launches);
cudaError_t launch_route_grad(const RouteJob &job, cudaStream_t stream, int *launches);

// Exclusive sums down the columns of tile_counts [tiles][bins], in place, and
// the columns' totals (expert.cu).
cudaError_t launch_tile_scan(uint32_t *tile_counts, uint32_t *totals, uint32_t tiles, uint32_t bins, cudaStream_t stream,
                             int *launches);

// The stable order of ids by table row, with their positions (id_order.cu).
struct IdOrderJob {
    const void *ids;
    int id_bytes;
    size_t n, vocab;
    int64_t first_id, padding_id;  // padding_id < 0: none
    Header *hdr;                   // ID_ORDER_CLEARED bytes from here are zeroed
    unsigned char *work;           // id_order_temp_bytes
    uint32_t *keys, *vals;         // out: sorted rows (vocab: none) and positions
};
constexpr size_t ID_ORDER_CLEARED = sizeof(Header) + 256;
size_t id_order_temp_bytes(size_t n, size_t vocab);
cudaError_t launch_id_order(const IdOrderJob &job, cudaStream_t stream, int *launches);

struct EmbeddingJob {
    const void *ids;
    int id_bytes;
    size_t n;
    int64_t first_id, padding_id;  // padding_id < 0: none
    size_t vocab, row_len;
    float scale;
    Rows table;  // lookup: the table; grad: its gradient
    Rows out;    // lookup: the rows; grad: the rows' gradient
    bool accumulate;
    unsigned char *temp;  // grad only: embedding_grad_temp_bytes
};
cudaError_t launch_embedding_lookup(const EmbeddingJob &job, cudaStream_t stream, int *launches);
// The test hook's chunk whose copies are held back (~0: none) and the tries of a
// wait for a copy (0: the default); see gbs_debug_set_ring_fault.
void debug_ring_settings(uint32_t *fault_chunk, uint32_t *spins);
size_t embedding_grad_temp_bytes(size_t n, size_t vocab, size_t row_len);
cudaError_t launch_embedding_grad(const EmbeddingJob &job, cudaStream_t stream, int *launches);

// A beam search's choice of its next beams (beam.cu).
struct BeamSelectJob {
    Rows logits;  // [batch * beams][vocab]
    size_t batch, vocab;
    uint32_t beams, num_out;
    const float *scores;
    const uint8_t *finished;  // nullptr: none
    int32_t end_id;
    unsigned char *temp;  // beam_select_temp_bytes
    float *scores_out;
    int32_t *beams_out, *tokens_out;
};
size_t beam_slices(size_t rows, size_t vocab, int type);
size_t beam_select_temp_bytes(size_t rows, size_t vocab, int type, size_t num_out);
cudaError_t launch_beam_select(const BeamSelectJob &job, cudaStream_t stream, int *launches);

// States [outer][batch][beams][segments][segment_bytes] by parent; strides in bytes.
struct BeamReorderJob {
    const unsigned char *in;
    unsigned char *out;  // in: in place
    size_t outer, batch, segments, segment_bytes;
    uint32_t beams, into;
    size_t in_outer, in_batch, in_beam, in_segment, out_outer, out_batch, out_beam, out_segment;
    const int32_t *parents;
};
cudaError_t launch_beam_reorder(const BeamReorderJob &job, cudaStream_t stream, int *launches);

}  // namespace gbs
