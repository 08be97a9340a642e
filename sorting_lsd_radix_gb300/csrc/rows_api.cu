// C ABI of the row operators: argument checks, work buffers, dispatch to the
// kernels of route.cu, expert.cu, embedding.cu and beam.cu.
#include <limits>

#include "../../include/gbsort.h"
#include "rows.h"

static_assert((int)GBS_ROW_F32 == gbs::ROW_F32 && (int)GBS_ROW_F16 == gbs::ROW_F16 && (int)GBS_ROW_BF16 == gbs::ROW_BF16,
              "the ABI's row types are the kernels' row types");

namespace {

using gbs::Header;
using gbs::Rows;

constexpr size_t ALIGN = 256;
constexpr size_t MAX_I32 = (size_t)std::numeric_limits<int32_t>::max();

bool is_row_type(int t) { return t == GBS_ROW_F32 || t == GBS_ROW_F16 || t == GBS_ROW_BF16; }
bool is_id_type(int t) { return t == GBS_I32 || t == GBS_I64; }
int id_bytes_of(int t) { return t == GBS_I64 ? 8 : 4; }
bool aligned(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Rows of `count` > 0 rows of `len` > 0 values that a kernel reads (stride 0:
// one row for all) or writes (rows apart from one another).
gbs_status check_rows(const Rows &r, size_t count, size_t len, bool written) {
    if (count == 0 || len == 0) return GBS_OK;
    if (r.base == nullptr || !aligned(r.base, (size_t)gbs::row_bytes(r.type))) return GBS_ERR_INVALID_ARG;
    if (written && count > 1 && r.stride < len) return GBS_ERR_INVALID_ARG;
    // the last row's last byte has an address
    const size_t most = std::numeric_limits<size_t>::max() / 8;
    if (count > 1 && r.stride > most / count) return GBS_ERR_UNSUPPORTED;
    return GBS_OK;
}

gbs_status check_temp(void *d_temp, size_t *temp_bytes, size_t need, bool *query) {
    *query = d_temp == nullptr;
    if (temp_bytes == nullptr) return GBS_ERR_INVALID_ARG;
    if (*query) {
        *temp_bytes = need;
        return GBS_OK;
    }
    if (!aligned(d_temp, ALIGN)) return GBS_ERR_INVALID_ARG;
    return *temp_bytes < need ? GBS_ERR_TEMP_TOO_SMALL : GBS_OK;
}

gbs_status from_cuda(cudaError_t e) { return e == cudaSuccess ? GBS_OK : GBS_ERR_CUDA; }

// The limits of a slot grid: GBS_ERR_INVALID_ARG or GBS_ERR_UNSUPPORTED outside them.
gbs_status check_slots(size_t num_tokens, size_t top_k, size_t num_rows, size_t row_len) {
    if (top_k == 0) return GBS_ERR_INVALID_ARG;
    if (top_k > GBS_MAX_TOP_K || row_len > GBS_MAX_ROW_LEN || num_rows > MAX_I32) return GBS_ERR_UNSUPPORTED;
    if (num_tokens > MAX_I32 / top_k) return GBS_ERR_UNSUPPORTED;
    return GBS_OK;
}

gbs_status dispatch(void *d_temp, size_t *temp_bytes, const Rows &x, const Rows &rows, size_t row_len, gbs_key_type id_type,
                    const void *d_expert_ids, size_t num_tokens, size_t top_k, size_t num_experts, int64_t first_expert,
                    size_t row_align, size_t num_rows, int32_t *d_slot_of_row, int32_t *d_row_of_slot, int32_t *d_offsets,
                    int32_t *d_counts, void *stream) {
    if (!is_id_type(id_type) || temp_bytes == nullptr) return GBS_ERR_INVALID_ARG;
    if (num_experts == 0 || row_align == 0) return GBS_ERR_INVALID_ARG;
    gbs_status st = check_slots(num_tokens, top_k, num_rows, row_len);
    if (st != GBS_OK) return st;
    if (num_experts > GBS_MAX_EXPERTS || row_align > GBS_MAX_ROW_LEN) return GBS_ERR_UNSUPPORTED;
    const size_t slots = num_tokens * top_k;
    if (gbs_expert_num_rows(slots, num_experts, row_align) > MAX_I32) return GBS_ERR_UNSUPPORTED;
    if (num_rows < gbs_expert_num_rows(slots, num_experts, row_align)) return GBS_ERR_INVALID_ARG;
    bool query = false;
    st = check_temp(d_temp, temp_bytes, sizeof(Header) + gbs::expert_temp_bytes(num_tokens, top_k, num_experts), &query);
    if (st != GBS_OK || query) return st;
    if (slots > 0 && (d_expert_ids == nullptr || d_row_of_slot == nullptr)) return GBS_ERR_INVALID_ARG;
    if (num_rows > 0 && d_slot_of_row == nullptr) return GBS_ERR_INVALID_ARG;
    if (d_offsets == nullptr || d_counts == nullptr) return GBS_ERR_INVALID_ARG;
    if (!aligned(d_expert_ids, (size_t)id_bytes_of(id_type)) || !aligned(d_slot_of_row, 4) || !aligned(d_row_of_slot, 4) ||
        !aligned(d_offsets, 4) || !aligned(d_counts, 4))
        return GBS_ERR_INVALID_ARG;
    gbs::ExpertJob job = {};
    job.ids = d_expert_ids;
    job.id_bytes = id_bytes_of(id_type);
    job.num_tokens = num_tokens;
    job.top_k = (uint32_t)top_k;
    job.num_experts = (uint32_t)num_experts;
    job.first_expert = first_expert;
    job.row_align = (uint32_t)row_align;
    job.num_rows = num_rows;
    job.slot_of_row = d_slot_of_row;
    job.row_of_slot = d_row_of_slot;
    job.offsets = d_offsets;
    job.counts = d_counts;
    job.hdr = static_cast<Header *>(d_temp);
    job.tile_counts = reinterpret_cast<uint32_t *>(static_cast<unsigned char *>(d_temp) + sizeof(Header));
    if (num_rows > 0) {
        job.x = x;
        job.rows = rows;
        job.row_len = row_len;
        // no token: the rows are only zeroed, and x is not read
        if (num_tokens == 0) job.x = rows;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(gbs::launch_expert_dispatch(job, s, gbs::call_begin(s)));
}

// That no place of a grid of four dimensions is there twice: ordered by stride, each
// dimension lies outside of what the ones before it cover.  And every place has an
// address.
gbs_status check_apart(const size_t *strides, const size_t *sizes, size_t bytes) {
    const size_t most = std::numeric_limits<size_t>::max() / 8;
    size_t covered = bytes;
    bool done[4] = {};
    for (int turn = 0; turn < 4; ++turn) {
        int next = -1;
        for (int i = 0; i < 4; ++i)
            if (!done[i] && (next < 0 || strides[i] < strides[next] || (strides[i] == strides[next] && sizes[i] < sizes[next])))
                next = i;
        done[next] = true;
        if (sizes[next] == 1) continue;
        if (strides[next] > (most - covered) / sizes[next]) return GBS_ERR_UNSUPPORTED;
        if (strides[next] < covered) return GBS_ERR_INVALID_ARG;
        covered += (sizes[next] - 1) * strides[next];
    }
    return GBS_OK;
}

// What route and its gradient share: GBS_OK with the job's logits, ids and
// weights in place, or the refusal.
gbs_status route_job(gbs::RouteJob *job, gbs_row_type row_type, const void *d_logits, size_t logits_stride, size_t num_tokens,
                     size_t num_experts, size_t top_k, gbs_score_type score_type, int renormalise, float scale,
                     gbs_key_type id_type, const void *d_expert_ids, gbs_row_type weight_type, const void *d_weights) {
    if (!is_row_type(row_type) || !is_id_type(id_type) || (weight_type != row_type && weight_type != GBS_ROW_F32))
        return GBS_ERR_INVALID_ARG;
    if (score_type != GBS_SCORE_SOFTMAX && score_type != GBS_SCORE_SIGMOID) return GBS_ERR_INVALID_ARG;
    if (num_experts == 0 || top_k == 0) return GBS_ERR_INVALID_ARG;
    if (num_experts > GBS_MAX_EXPERTS || top_k > GBS_MAX_TOP_K || num_tokens > MAX_I32 / top_k) return GBS_ERR_UNSUPPORTED;
    if (top_k > num_experts) return GBS_ERR_INVALID_ARG;
    job->logits = {const_cast<void *>(d_logits), logits_stride, row_type};
    const gbs_status st = check_rows(job->logits, num_tokens, num_experts, false);
    if (st != GBS_OK) return st;
    if (num_tokens > 0 && (d_expert_ids == nullptr || d_weights == nullptr)) return GBS_ERR_INVALID_ARG;
    if (!aligned(d_expert_ids, (size_t)id_bytes_of(id_type)) || !aligned(d_weights, (size_t)gbs::row_bytes(weight_type)))
        return GBS_ERR_INVALID_ARG;
    job->num_tokens = num_tokens;
    job->num_experts = (uint32_t)num_experts;
    job->top_k = (uint32_t)top_k;
    job->sigmoid = score_type == GBS_SCORE_SIGMOID;
    job->renormalise = renormalise != 0;
    job->scale = scale;
    job->ids = const_cast<void *>(d_expert_ids);
    job->id_bytes = id_bytes_of(id_type);
    job->weights = const_cast<void *>(d_weights);
    job->weight_type = weight_type;
    return GBS_OK;
}

}  // namespace

extern "C" {

size_t gbs_expert_num_rows(size_t num_slots, size_t num_experts, size_t row_align) {
    if (row_align <= 1) return num_slots;
    const size_t used = num_slots < num_experts ? num_slots : num_experts;
    if (used > 0 && row_align - 1 > (std::numeric_limits<size_t>::max() - num_slots) / used)
        return std::numeric_limits<size_t>::max();
    return (num_slots + used * (row_align - 1)) / row_align * row_align;
}

gbs_status gbs_expert_sort(void *d_temp, size_t *temp_bytes, gbs_key_type id_type, const void *d_expert_ids,
                           size_t num_tokens, size_t top_k, size_t num_experts, int64_t first_expert, size_t row_align,
                           size_t num_rows, int32_t *d_slot_of_row, int32_t *d_row_of_slot, int32_t *d_offsets,
                           int32_t *d_counts, void *stream) {
    const Rows none = {nullptr, 0, GBS_ROW_F32};
    return dispatch(d_temp, temp_bytes, none, none, 0, id_type, d_expert_ids, num_tokens, top_k, num_experts,
                    first_expert, row_align, num_rows, d_slot_of_row, d_row_of_slot, d_offsets, d_counts, stream);
}

gbs_status gbs_expert_dispatch(void *d_temp, size_t *temp_bytes, gbs_row_type row_type, const void *d_x, size_t x_stride,
                               size_t row_len, gbs_key_type id_type, const void *d_expert_ids, size_t num_tokens,
                               size_t top_k, size_t num_experts, int64_t first_expert, size_t row_align, size_t num_rows,
                               void *d_rows, size_t rows_stride, int32_t *d_slot_of_row, int32_t *d_row_of_slot,
                               int32_t *d_offsets, int32_t *d_counts, void *stream) {
    if (!is_row_type(row_type)) return GBS_ERR_INVALID_ARG;
    const Rows x = {const_cast<void *>(d_x), x_stride, row_type}, rows = {d_rows, rows_stride, row_type};
    if (d_temp != nullptr) {
        gbs_status st = check_rows(x, num_tokens, row_len, false);
        if (st == GBS_OK) st = check_rows(rows, num_rows, row_len, true);
        if (st != GBS_OK) return st;
    }
    return dispatch(d_temp, temp_bytes, x, rows, row_len, id_type, d_expert_ids, num_tokens, top_k, num_experts,
                    first_expert, row_align, num_rows, d_slot_of_row, d_row_of_slot, d_offsets, d_counts, stream);
}

gbs_status gbs_expert_gather(gbs_row_type row_type, const void *d_x, size_t x_stride, size_t num_tokens, size_t top_k,
                             size_t row_len, const int32_t *d_slot_of_row, const int32_t *d_row_of_slot, size_t num_rows,
                             void *d_rows, size_t rows_stride, void *stream) {
    if (!is_row_type(row_type)) return GBS_ERR_INVALID_ARG;
    gbs_status st = check_slots(num_tokens, top_k, num_rows, row_len);
    if (st != GBS_OK) return st;
    gbs::ExpertMoveJob job = {};
    job.x = {const_cast<void *>(d_x), x_stride, row_type};
    job.rows = {d_rows, rows_stride, row_type};
    st = check_rows(job.x, num_tokens, row_len, false);
    if (st == GBS_OK) st = check_rows(job.rows, num_rows, row_len, true);
    if (st != GBS_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int *launches = gbs::call_begin(s);
    if (num_rows == 0 || row_len == 0) return GBS_OK;
    if (d_slot_of_row == nullptr || (num_tokens > 0 && d_row_of_slot == nullptr)) return GBS_ERR_INVALID_ARG;
    if (!aligned(d_slot_of_row, 4) || !aligned(d_row_of_slot, 4)) return GBS_ERR_INVALID_ARG;
    if (num_tokens == 0) job.x = job.rows;
    job.slot_of_row = d_slot_of_row;
    job.row_of_slot = d_row_of_slot;
    job.num_tokens = num_tokens;
    job.num_rows = num_rows;
    job.row_len = row_len;
    job.top_k = (uint32_t)top_k;
    return from_cuda(gbs::launch_expert_gather(job, s, launches));
}

gbs_status gbs_expert_combine(gbs_row_type row_type, const void *d_rows, size_t rows_stride, size_t num_rows,
                              const int32_t *d_row_of_slot, gbs_row_type weight_type, const void *d_weights,
                              size_t num_tokens, size_t top_k, size_t row_len, void *d_out, size_t out_stride,
                              void *stream) {
    if (!is_row_type(row_type)) return GBS_ERR_INVALID_ARG;
    if (d_weights != nullptr && weight_type != row_type && weight_type != GBS_ROW_F32) return GBS_ERR_INVALID_ARG;
    gbs_status st = check_slots(num_tokens, top_k, num_rows, row_len);
    if (st != GBS_OK) return st;
    gbs::ExpertMoveJob job = {};
    job.x = {d_out, out_stride, row_type};
    job.rows = {const_cast<void *>(d_rows), rows_stride, row_type};
    st = check_rows(job.x, num_tokens, row_len, true);
    if (st == GBS_OK) st = check_rows(job.rows, num_rows, row_len, false);
    if (st != GBS_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int *launches = gbs::call_begin(s);
    if (num_tokens == 0 || row_len == 0) return GBS_OK;
    if (d_row_of_slot == nullptr || !aligned(d_row_of_slot, 4)) return GBS_ERR_INVALID_ARG;
    if (d_weights != nullptr && !aligned(d_weights, (size_t)gbs::row_bytes(weight_type))) return GBS_ERR_INVALID_ARG;
    if (num_rows == 0) job.rows = job.x;  // every slot is without a row: nothing is read
    job.row_of_slot = d_row_of_slot;
    job.num_tokens = num_tokens;
    job.num_rows = num_rows;
    job.row_len = row_len;
    job.top_k = (uint32_t)top_k;
    job.weight_type = d_weights != nullptr ? weight_type : GBS_ROW_F32;
    job.weights = d_weights;
    return from_cuda(gbs::launch_expert_combine(job, s, launches));
}

gbs_status gbs_expert_combine_grad(gbs_row_type row_type, const void *d_dout, size_t dout_stride, const void *d_rows,
                                   size_t rows_stride, size_t num_rows, const int32_t *d_slot_of_row,
                                   const int32_t *d_row_of_slot, gbs_row_type weight_type, const void *d_weights,
                                   size_t num_tokens, size_t top_k, size_t row_len, void *d_drows, size_t drows_stride,
                                   void *d_dweights, void *stream) {
    if (!is_row_type(row_type)) return GBS_ERR_INVALID_ARG;
    const bool weighted = d_weights != nullptr || d_dweights != nullptr;
    if (weighted && weight_type != row_type && weight_type != GBS_ROW_F32) return GBS_ERR_INVALID_ARG;
    gbs_status st = check_slots(num_tokens, top_k, num_rows, row_len);
    if (st != GBS_OK) return st;
    gbs::ExpertMoveJob job = {};
    job.x = {const_cast<void *>(d_dout), dout_stride, row_type};
    job.rows = {const_cast<void *>(d_rows), rows_stride, row_type};
    job.d_rows = {d_drows, drows_stride, row_type};
    st = check_rows(job.x, num_tokens, row_len, false);
    if (st == GBS_OK && d_dweights != nullptr) st = check_rows(job.rows, num_rows, row_len, false);
    if (st == GBS_OK) st = check_rows(job.d_rows, num_rows, row_len, true);
    if (st != GBS_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int *launches = gbs::call_begin(s);
    if (num_tokens == 0 && num_rows == 0) return GBS_OK;
    if ((num_rows > 0 && d_slot_of_row == nullptr) || (num_tokens > 0 && d_row_of_slot == nullptr)) return GBS_ERR_INVALID_ARG;
    if (!aligned(d_slot_of_row, 4) || !aligned(d_row_of_slot, 4)) return GBS_ERR_INVALID_ARG;
    if (weighted && (!aligned(d_weights, (size_t)gbs::row_bytes(weight_type)) ||
                     !aligned(d_dweights, (size_t)gbs::row_bytes(weight_type))))
        return GBS_ERR_INVALID_ARG;
    if (num_tokens == 0) job.x = job.d_rows;
    if (num_rows == 0) job.d_rows = job.x;
    if (num_rows == 0 || d_dweights == nullptr) job.rows = job.d_rows;  // not read
    job.slot_of_row = d_slot_of_row;
    job.row_of_slot = d_row_of_slot;
    job.num_tokens = num_tokens;
    job.num_rows = num_rows;
    job.row_len = row_len;
    job.top_k = (uint32_t)top_k;
    job.weight_type = weighted ? weight_type : GBS_ROW_F32;
    job.weights = d_weights;
    job.d_weights = d_dweights;
    return from_cuda(gbs::launch_expert_combine_grad(job, s, launches));
}

gbs_status gbs_expert_route(gbs_row_type row_type, const void *d_logits, size_t logits_stride, size_t num_tokens,
                            size_t num_experts, size_t top_k, gbs_score_type score_type, const float *d_bias,
                            size_t num_groups, size_t top_groups, size_t group_top, int renormalise, float scale,
                            gbs_key_type id_type, void *d_expert_ids, gbs_row_type weight_type, void *d_weights,
                            void *stream) {
    gbs::RouteJob job = {};
    const gbs_status st = route_job(&job, row_type, d_logits, logits_stride, num_tokens, num_experts, top_k, score_type,
                                    renormalise, scale, id_type, d_expert_ids, weight_type, d_weights);
    if (st != GBS_OK) return st;
    if (num_groups == 0 || num_experts % num_groups != 0 || top_groups == 0 || top_groups > num_groups)
        return GBS_ERR_INVALID_ARG;
    if (group_top != 1 && group_top != 2) return GBS_ERR_INVALID_ARG;
    if (num_groups > GBS_MAX_GROUPS) return GBS_ERR_UNSUPPORTED;
    if (top_k > top_groups * (num_experts / num_groups)) return GBS_ERR_INVALID_ARG;
    if (!aligned(d_bias, 4)) return GBS_ERR_INVALID_ARG;
    job.bias = d_bias;
    job.num_groups = (uint32_t)num_groups;
    job.top_groups = (uint32_t)top_groups;
    job.group_top = (uint32_t)group_top;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(gbs::launch_route(job, s, gbs::call_begin(s)));
}

gbs_status gbs_expert_route_grad(gbs_row_type row_type, gbs_row_type weight_type, const void *d_dweights,
                                 const void *d_logits, size_t logits_stride, size_t num_tokens, size_t num_experts,
                                 size_t top_k, gbs_key_type id_type, const void *d_expert_ids, gbs_score_type score_type,
                                 int renormalise, float scale, void *d_dlogits, size_t dlogits_stride, void *stream) {
    gbs::RouteJob job = {};
    gbs_status st = route_job(&job, row_type, d_logits, logits_stride, num_tokens, num_experts, top_k, score_type,
                              renormalise, scale, id_type, d_expert_ids, weight_type, d_dweights);
    if (st != GBS_OK) return st;
    job.d_logits = {d_dlogits, dlogits_stride, row_type};
    st = check_rows(job.d_logits, num_tokens, num_experts, true);
    if (st != GBS_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(gbs::launch_route_grad(job, s, gbs::call_begin(s)));
}

gbs_status gbs_embedding_lookup(gbs_row_type row_type, const void *d_table, size_t table_stride, size_t vocab,
                                gbs_key_type id_type, const void *d_ids, size_t n, int64_t first_id, float scale,
                                size_t row_len, void *d_out, size_t out_stride, void *stream) {
    if (!is_row_type(row_type) || !is_id_type(id_type)) return GBS_ERR_INVALID_ARG;
    if (n > MAX_I32 || vocab > MAX_I32 - 1 || row_len > GBS_MAX_ROW_LEN) return GBS_ERR_UNSUPPORTED;
    gbs::EmbeddingJob job = {};
    job.table = {const_cast<void *>(d_table), table_stride, row_type};
    job.out = {d_out, out_stride, row_type};
    gbs_status st = check_rows(job.table, n > 0 ? vocab : 0, row_len, false);
    if (st == GBS_OK) st = check_rows(job.out, n, row_len, true);
    if (st != GBS_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int *launches = gbs::call_begin(s);
    if (n == 0 || row_len == 0) return GBS_OK;
    if (d_ids == nullptr || !aligned(d_ids, (size_t)id_bytes_of(id_type))) return GBS_ERR_INVALID_ARG;
    if (vocab == 0) job.table = job.out;  // every id is outside: nothing is read
    job.ids = d_ids;
    job.id_bytes = id_bytes_of(id_type);
    job.n = n;
    job.first_id = first_id;
    job.vocab = vocab;
    job.row_len = row_len;
    job.scale = scale;
    return from_cuda(gbs::launch_embedding_lookup(job, s, launches));
}

gbs_status gbs_embedding_grad(void *d_temp, size_t *temp_bytes, gbs_row_type row_type, const void *d_dout,
                              size_t dout_stride, gbs_key_type id_type, const void *d_ids, size_t n, int64_t first_id,
                              int64_t padding_id, float scale, size_t vocab, size_t row_len, gbs_row_type grad_type,
                              void *d_grad, size_t grad_stride, int accumulate, void *stream) {
    if (!is_row_type(row_type) || !is_row_type(grad_type) || !is_id_type(id_type)) return GBS_ERR_INVALID_ARG;
    if (grad_type != row_type && grad_type != GBS_ROW_F32) return GBS_ERR_INVALID_ARG;
    if (temp_bytes == nullptr) return GBS_ERR_INVALID_ARG;
    if (n > MAX_I32 || vocab > MAX_I32 - 1 || row_len > GBS_MAX_ROW_LEN) return GBS_ERR_UNSUPPORTED;
    bool query = false;
    gbs_status st = check_temp(d_temp, temp_bytes, gbs::embedding_grad_temp_bytes(n, vocab, row_len), &query);
    if (st != GBS_OK || query) return st;
    gbs::EmbeddingJob job = {};
    job.out = {const_cast<void *>(d_dout), dout_stride, row_type};
    job.table = {d_grad, grad_stride, grad_type};
    st = check_rows(job.out, n, row_len, false);
    if (st == GBS_OK) st = check_rows(job.table, vocab, row_len, true);
    if (st != GBS_OK) return st;
    if (n > 0 && (d_ids == nullptr || !aligned(d_ids, (size_t)id_bytes_of(id_type)))) return GBS_ERR_INVALID_ARG;
    job.ids = d_ids;
    job.id_bytes = id_bytes_of(id_type);
    job.n = n;
    job.first_id = first_id;
    job.padding_id = padding_id;
    job.vocab = vocab;
    job.row_len = row_len;
    job.scale = scale;
    job.accumulate = accumulate != 0;
    job.temp = static_cast<unsigned char *>(d_temp);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(gbs::launch_embedding_grad(job, s, gbs::call_begin(s)));
}

gbs_status gbs_beam_select(void *d_temp, size_t *temp_bytes, gbs_row_type row_type, const void *d_logits,
                           size_t logits_stride, size_t batch, size_t beams, size_t vocab, const float *d_scores,
                           const uint8_t *d_finished, int32_t end_id, size_t num_out, float *d_scores_out,
                           int32_t *d_beams_out, int32_t *d_tokens_out, void *stream) {
    if (!is_row_type(row_type) || temp_bytes == nullptr) return GBS_ERR_INVALID_ARG;
    if (beams == 0 || vocab == 0 || num_out == 0) return GBS_ERR_INVALID_ARG;
    if (beams > GBS_MAX_BEAMS || num_out > GBS_MAX_BEAM_OUT || vocab > MAX_I32 || batch > MAX_I32 / beams) return GBS_ERR_UNSUPPORTED;
    const size_t rows = batch * beams;
    if (rows > 0 && gbs::beam_slices(rows, vocab, row_type) > MAX_I32 / rows) return GBS_ERR_UNSUPPORTED;
    bool query = false;
    gbs_status st = check_temp(d_temp, temp_bytes, gbs::beam_select_temp_bytes(rows, vocab, row_type, num_out), &query);
    if (st != GBS_OK || query) return st;
    gbs::BeamSelectJob job = {};
    job.logits = {const_cast<void *>(d_logits), logits_stride, row_type};
    st = check_rows(job.logits, rows, vocab, false);
    if (st != GBS_OK) return st;
    if (rows > 0 && (d_scores == nullptr || d_scores_out == nullptr || d_beams_out == nullptr || d_tokens_out == nullptr))
        return GBS_ERR_INVALID_ARG;
    if (!aligned(d_scores, 4) || !aligned(d_scores_out, 4) || !aligned(d_beams_out, 4) || !aligned(d_tokens_out, 4))
        return GBS_ERR_INVALID_ARG;
    job.batch = batch;
    job.vocab = vocab;
    job.beams = (uint32_t)beams;
    job.num_out = (uint32_t)num_out;
    job.scores = d_scores;
    job.finished = d_finished;
    job.end_id = end_id;
    job.temp = static_cast<unsigned char *>(d_temp);
    job.scores_out = d_scores_out;
    job.beams_out = d_beams_out;
    job.tokens_out = d_tokens_out;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(gbs::launch_beam_select(job, s, gbs::call_begin(s)));
}

gbs_status gbs_beam_reorder(const void *d_in, const size_t *in_strides, void *d_out, const size_t *out_strides, size_t outer,
                            size_t batch, size_t in_beams, size_t out_beams, size_t segments, size_t segment_bytes,
                            const int32_t *d_parents, void *stream) {
    if (in_strides == nullptr || out_strides == nullptr) return GBS_ERR_INVALID_ARG;
    if (in_beams > GBS_MAX_BEAMS || out_beams > GBS_MAX_BEAMS) return GBS_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (outer == 0 || batch == 0 || out_beams == 0 || segments == 0 || segment_bytes == 0) {
        gbs::call_begin(s);
        return GBS_OK;
    }
    if (in_beams == 0) return GBS_ERR_INVALID_ARG;
    if (batch > MAX_I32 || segments > MAX_I32 / batch || segment_bytes > MAX_I32 / (batch * segments)) return GBS_ERR_UNSUPPORTED;
    if (d_in == nullptr || d_out == nullptr || d_parents == nullptr || !aligned(d_parents, 4)) return GBS_ERR_INVALID_ARG;
    const size_t writes[4] = {outer, batch, out_beams, segments}, reads[4] = {outer, batch, in_beams, segments};
    for (int i = 0; i < 4; ++i)
        if (reads[i] > 1 && in_strides[i] > std::numeric_limits<size_t>::max() / 8 / reads[i]) return GBS_ERR_UNSUPPORTED;
    gbs_status st = check_apart(out_strides, writes, segment_bytes);
    if (st != GBS_OK) return st;
    if (d_in == d_out) {
        if (out_beams > in_beams) return GBS_ERR_INVALID_ARG;
        for (int i = 0; i < 4; ++i)
            if (writes[i] > 1 && in_strides[i] != out_strides[i]) return GBS_ERR_INVALID_ARG;
        // a beam that is only read must not be another batch's that is written
        st = check_apart(in_strides, reads, segment_bytes);
        if (st != GBS_OK) return st;
    }
    gbs::BeamReorderJob job = {};
    job.in = static_cast<const unsigned char *>(d_in);
    job.out = static_cast<unsigned char *>(d_out);
    job.outer = outer;
    job.batch = batch;
    job.segments = segments;
    job.segment_bytes = segment_bytes;
    job.beams = (uint32_t)in_beams;
    job.into = (uint32_t)out_beams;
    // a dimension of one has no stride
    job.in_outer = outer > 1 ? in_strides[0] : 0;
    job.in_batch = batch > 1 ? in_strides[1] : 0;
    job.in_beam = in_beams > 1 ? in_strides[2] : 0;
    job.in_segment = segments > 1 ? in_strides[3] : 0;
    job.out_outer = outer > 1 ? out_strides[0] : 0;
    job.out_batch = batch > 1 ? out_strides[1] : 0;
    job.out_beam = out_beams > 1 ? out_strides[2] : 0;
    job.out_segment = segments > 1 ? out_strides[3] : 0;
    job.parents = d_parents;
    return from_cuda(gbs::launch_beam_reorder(job, s, gbs::call_begin(s)));
}

}  // extern "C"
