// C ABI of the row operators: argument checks, work buffers, dispatch to the
// kernels of expert.cu and embedding.cu.
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

}  // extern "C"
