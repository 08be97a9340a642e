// Embedding rows looked up by token id, and the table's gradient.
//
//   lookup    out[i] = scale * table[ids[i] - first_id], zeros where the id
//             is outside the table (a shard of a vocabulary)
//   gradient  grad[v] (+)= scale * sum of d_out[i] over ids[i] - first_id = v
//
// The gradient sorts (id, i) stably by id with the library's radix sort, so
// that each table row's terms are neighbours, in the order of i.  The sorted
// positions are cut into chunks of equal length; a CTA sums the runs of equal
// ids of its chunk in 32 bits.  A run inside one chunk goes to the table at
// once; one that crosses a chunk's end leaves 32-bit partial sums, which a
// second kernel adds in the order of the chunks.  No atomics touch a sum, so
// equal inputs give equal bits.  Both directions are bound by bytes: one
// addition per value read.
#include "rows.cuh"

namespace gbs {
namespace {

constexpr int ROW_THREADS = 256;

struct LookupParams {
    const void *ids;
    int id_bytes;
    int64_t first;
    uint64_t n, vocab;
    const unsigned char *table;
    unsigned char *out;
    size_t table_stride, out_stride;  // bytes
    uint32_t row_len;
    float scale;
};

// threadIdx.x: packs of N columns; threadIdx.y: an id.
template <typename T, int N> __global__ void __launch_bounds__(ROW_THREADS) embedding_lookup_kernel(const LookupParams p) {
    const uint64_t i = (uint64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (i >= p.n) return;
    const int32_t at = id_index(p.ids, p.id_bytes, i, p.first, p.vocab);
    const T *src = reinterpret_cast<const T *>(p.table + (size_t)(at < 0 ? 0 : at) * p.table_stride);
    T *dst = reinterpret_cast<T *>(p.out + i * p.out_stride);
    constexpr int U = 4;
    const uint32_t step = gridDim.y * blockDim.x * N;
    for (uint32_t c0 = (blockIdx.y * blockDim.x + threadIdx.x) * N; c0 < p.row_len; c0 += step * U) {
        Pack<T, N> v[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            v[j] = Pack<T, N>{};
            if (at >= 0 && c0 + step * j < p.row_len) v[j] = load_pack<T, N>(src + c0 + step * j);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (p.scale != 1.0f)
#pragma unroll
                for (int k = 0; k < N; ++k) v[j].v[k] = at < 0 ? T{} : from_f32<T>(p.scale * to_f32(v[j].v[k]));
            if (c0 + step * j < p.row_len) store_pack(dst + c0 + step * j, v[j]);
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------

// Sort keys: the table row of each id, `vocab` (sorted last) for ids that
// have none; values: the position.
__global__ void __launch_bounds__(256) embedding_keys_kernel(const void *ids, int id_bytes, uint64_t n, int64_t first,
                                                             int64_t padding, uint32_t vocab, uint32_t *keys,
                                                             uint32_t *vals) {
    const uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    int32_t at = id_index(ids, id_bytes, i, first, vocab);
    if (padding >= 0) {
        const int64_t id = id_bytes == 8 ? static_cast<const int64_t *>(ids)[i] : static_cast<const int32_t *>(ids)[i];
        if (id == padding) at = -1;
    }
    keys[i] = at < 0 ? vocab : (uint32_t)at;
    vals[i] = (uint32_t)i;
}

struct GradParams {
    const uint32_t *keys, *vals;  // sorted
    uint32_t n, vocab, chunk, chunks;
    const unsigned char *d_out;
    unsigned char *grad;
    size_t d_out_stride, grad_stride;  // bytes
    uint32_t row_len;
    float scale;
    int accumulate;
    float *partial;      // [2 * chunks][row_len]: a chunk's run from the chunk before, its run into the next
    uint32_t *crossing;  // chunks whose last run goes on and starts in them, any order
    uint32_t *crossings; // how many
};

constexpr uint32_t CHUNK_MOST = 64;

template <typename G, int N> __device__ __forceinline__ void to_table(G *dst, const float *acc, float scale, int accumulate,
                                                                      const Pack<G, N> &old) {
    Pack<G, N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.v[i] = from_f32<G>(accumulate ? fmaf(scale, acc[i], to_f32(old.v[i])) : scale * acc[i]);
    store_pack(dst, o);
}

// A CTA sums one chunk of sorted positions, a pack of N columns per thread.
template <typename T, typename G, int N> __global__ void __launch_bounds__(ROW_THREADS) embedding_sum_kernel(const GradParams p) {
    __shared__ uint32_t key[CHUNK_MOST + 2], val[CHUNK_MOST];
    const uint32_t b = blockIdx.x * p.chunk, len = min(p.chunk, p.n - b);
    // key[1 + j]: position b + j; key[0] and key[len + 1]: the neighbours (vocab + 1 where there is none).
    // A sort that timed out (reported by the header) leaves any values: none is followed outside d_out.
    for (uint32_t j = threadIdx.x; j < len + 2; j += blockDim.x) {
        const int64_t at = (int64_t)b + j - 1;
        key[j] = at >= 0 && at < p.n ? p.keys[at] : p.vocab + 1;
        if (j >= 1 && j <= len) {
            val[j - 1] = p.vals[at];
            if (val[j - 1] >= p.n) key[j] = p.vocab;
        }
    }
    __syncthreads();
    if (blockIdx.y == 0 && threadIdx.x == 0) {
        const uint32_t last = key[len];
        if (last < p.vocab && key[len + 1] == last && !(key[0] == last && key[1] == last))
            p.crossing[atomicAdd(p.crossings, 1u)] = blockIdx.x;
    }
    const uint32_t c = (blockIdx.y * blockDim.x + threadIdx.x) * N;
    if (c >= p.row_len) return;
    float acc[N] = {};
    constexpr uint32_t U = 4;
    bool from_before = key[0] == key[1];
    for (uint32_t j0 = 0; j0 < len; j0 += U) {
        Pack<T, N> v[U];
        Pack<G, N> old[U];
        // a run that ends at j0 + j inside this chunk is written at once
#pragma unroll
        for (uint32_t j = 0; j < U; ++j) {
            v[j] = Pack<T, N>{};
            old[j] = Pack<G, N>{};
            if (j0 + j < len && key[1 + j0 + j] < p.vocab) {
                v[j] = load_pack<T, N>(reinterpret_cast<const T *>(p.d_out + val[j0 + j] * p.d_out_stride) + c);
                if (p.accumulate && key[2 + j0 + j] != key[1 + j0 + j])
                    old[j] = load_pack<G, N>(reinterpret_cast<const G *>(p.grad + key[1 + j0 + j] * p.grad_stride) + c);
            }
        }
#pragma unroll
        for (uint32_t j = 0; j < U; ++j) {
            if (j0 + j >= len || key[1 + j0 + j] >= p.vocab) break;
            const uint32_t k = key[1 + j0 + j];
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] += to_f32(v[j].v[i]);
            const bool ends = key[2 + j0 + j] != k;
            if (ends && !from_before) {
                to_table<G, N>(reinterpret_cast<G *>(p.grad + k * p.grad_stride) + c, acc, p.scale, p.accumulate, old[j]);
            } else if (ends || j0 + j + 1 == len) {
                Pack<float, N> sum;
#pragma unroll
                for (int i = 0; i < N; ++i) sum.v[i] = acc[i];
                store_pack(p.partial + (2 * (size_t)blockIdx.x + (from_before ? 0 : 1)) * p.row_len + c, sum);
            }
            if (ends) {
                from_before = false;
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] = 0.0f;
            }
        }
    }
}

// Adds the partial sums of the runs that cross a chunk's end: an item is one
// such run and 32 packs of columns.  The warps share the run's chunks, each
// in order, and the CTA adds the warps' sums in order.
template <typename G, int N> __global__ void __launch_bounds__(ROW_THREADS) embedding_join_kernel(const GradParams p) {
    constexpr int WARPS = ROW_THREADS / 32;
    __shared__ float sums[WARPS][32 * N + 1];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t blocks = (p.row_len + 32 * N - 1) / (32 * N);
    const uint64_t items = (uint64_t)*p.crossings * blocks;
    for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const uint32_t chunk = p.crossing[it / blocks], c = (uint32_t)(it % blocks) * 32 * N + lane * N;
        const uint32_t k = p.keys[(size_t)(chunk + 1) * p.chunk];
        // the last chunk that begins with this run
        uint32_t lo = chunk + 1, hi = p.chunks - 1;
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo + 1) / 2;
            if (p.keys[(size_t)mid * p.chunk] == k) lo = mid;
            else hi = mid - 1;
        }
        float acc[N] = {};
        if (c < p.row_len) {
#pragma unroll 4
            for (uint32_t q = chunk + warp; q <= lo; q += WARPS) {
                const Pack<float, N> sum = load_pack<float, N>(p.partial + (2 * (size_t)q + (q == chunk ? 1 : 0)) * p.row_len + c);
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] += sum.v[i];
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) sums[warp][lane * N + i] = acc[i];
        __syncthreads();
        if (warp == 0 && c < p.row_len) {
            for (int w = 1; w < WARPS; ++w)
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] += sums[w][lane * N + i];
            G *dst = reinterpret_cast<G *>(p.grad + k * p.grad_stride) + c;
            Pack<G, N> old = Pack<G, N>{};
            if (p.accumulate) old = load_pack<G, N>(dst);
            to_table<G, N>(dst, acc, p.scale, p.accumulate, old);
        }
        __syncthreads();
    }
}

// Zeroes a table of rows; a thread takes packs of 16 bytes or less.
template <typename WORD> __global__ void __launch_bounds__(256) zero_rows_kernel(unsigned char *rows, size_t stride, uint64_t count,
                                                                                 uint32_t words) {
    const uint64_t total = count * words;
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (uint64_t)gridDim.x * 256)
        reinterpret_cast<WORD *>(rows + i / words * stride)[i % words] = WORD{};
}

uint32_t chunk_of(size_t n, size_t row_len) {
    (void)n;
    (void)row_len;
    return 32;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

struct GradLayout {
    size_t hist, base, status, keys, vals, keys_sorted, vals_sorted, keys_alt, vals_alt, crossings, crossing, partial, total;
    uint32_t tiles, chunks;
};
GradLayout grad_layout(size_t n, size_t row_len) {
    GradLayout l;
    const uint32_t tile = radix_tile_keys(4, 4);
    l.tiles = (uint32_t)((n + tile - 1) / tile);
    const size_t chunk = chunk_of(n, row_len);
    l.chunks = (uint32_t)((n + chunk - 1) / chunk);
    const size_t hist = up(sizeof(uint32_t) * MAX_PASSES * 256), list = up(sizeof(uint32_t) * n);
    size_t off = sizeof(Header);
    l.hist = off;
    l.crossings = off += hist;
    l.base = off += 256;
    l.status = off += hist;
    l.keys = off += up(status_bytes(n, l.tiles));
    l.vals = off += list;
    l.keys_sorted = off += list;
    l.vals_sorted = off += list;
    l.keys_alt = off += list;
    l.vals_alt = off += list;
    l.crossing = off += list;
    l.partial = off += up(sizeof(uint32_t) * (size_t)l.chunks);
    l.total = off + up(sizeof(float) * 2 * l.chunks * row_len);
    return l;
}

template <typename T, typename G, int N> cudaError_t launch_sums(const GradParams &p, cudaStream_t stream, int *launches) {
    const uint32_t packs = p.row_len / N;
    uint32_t threads = 32;
    while (threads < packs && threads < ROW_THREADS) threads *= 2;
    const dim3 grid(p.chunks, (packs + threads - 1) / threads);
    embedding_sum_kernel<T, G, N><<<grid, threads, 0, stream>>>(p);
    ++*launches;
    timing_mark(stream);
    if (p.chunks > 1) {
        embedding_join_kernel<G, N><<<(unsigned)device_sm_count() * 4, ROW_THREADS, 0, stream>>>(p);
        ++*launches;
        timing_mark(stream);
    }
    return cudaGetLastError();
}

template <typename T, typename G> cudaError_t launch_sums_by_width(const GradParams &p, int n, cudaStream_t stream, int *launches) {
    constexpr int FULL = 16 / (int)sizeof(T);
    if (n >= FULL) return launch_sums<T, G, FULL>(p, stream, launches);
    if (n >= 2) return launch_sums<T, G, 2>(p, stream, launches);
    return launch_sums<T, G, 1>(p, stream, launches);
}

template <typename T> cudaError_t launch_sums_by_grad(const GradParams &p, int type, int n, cudaStream_t stream, int *launches) {
    if (type == ROW_F32) return launch_sums_by_width<T, float>(p, n, stream, launches);
    return launch_sums_by_width<T, T>(p, n, stream, launches);
}

template <typename T, int N> cudaError_t launch_lookup(const LookupParams &p, cudaStream_t stream) {
    const uint32_t packs = p.row_len / N;
    uint32_t tx = 32;
    while (tx < packs && tx < ROW_THREADS) tx *= 2;
    const uint32_t ty = ROW_THREADS / tx, blocks = (uint32_t)((p.n + ty - 1) / ty);
    uint32_t cols = (packs + tx - 1) / tx;
    if (cols > 1 && blocks >= 4 * (uint32_t)device_sm_count()) cols = 1;
    embedding_lookup_kernel<T, N><<<dim3(blocks, cols), dim3(tx, ty), 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_lookup_by_width(const LookupParams &p, int n, cudaStream_t stream) {
    constexpr int FULL = 16 / (int)sizeof(T);
    if (n >= FULL) return launch_lookup<T, FULL>(p, stream);
    if (n >= 2) return launch_lookup<T, 2>(p, stream);
    return launch_lookup<T, 1>(p, stream);
}

}  // namespace

cudaError_t launch_embedding_lookup(const EmbeddingJob &job, cudaStream_t stream, int *launches) {
    LookupParams p = {};
    const size_t b = (size_t)row_bytes(job.table.type);
    p.ids = job.ids;
    p.id_bytes = job.id_bytes;
    p.first = job.first_id;
    p.n = job.n;
    p.vocab = job.vocab;
    p.table = static_cast<const unsigned char *>(job.table.base);
    p.out = static_cast<unsigned char *>(job.out.base);
    p.table_stride = job.table.stride * b;
    p.out_stride = job.out.stride * b;
    p.row_len = (uint32_t)job.row_len;
    p.scale = job.scale;
    const Rows rows[2] = {job.table, job.out};
    const int n = pack_values(rows, 2, job.row_len);
    const cudaError_t e = job.table.type == ROW_F32   ? launch_lookup_by_width<float>(p, n, stream)
                          : job.table.type == ROW_F16 ? launch_lookup_by_width<__half>(p, n, stream)
                                                      : launch_lookup_by_width<__nv_bfloat16>(p, n, stream);
    ++*launches;
    timing_mark(stream);
    return e;
}

size_t embedding_grad_temp_bytes(size_t n, size_t vocab, size_t row_len) {
    (void)vocab;
    return grad_layout(n, row_len).total;
}

cudaError_t launch_embedding_grad(const EmbeddingJob &job, cudaStream_t stream, int *launches) {
    const GradLayout lay = grad_layout(job.n, job.row_len);
    unsigned char *t = job.temp;
    const size_t gb = (size_t)row_bytes(job.table.type), db = (size_t)row_bytes(job.out.type);
    cudaError_t e = cudaMemsetAsync(t, 0, lay.base, stream);  // header, histograms, the count of crossing runs
    if (e != cudaSuccess) return e;
    if (!job.accumulate && job.vocab > 0 && job.row_len > 0) {
        const int n = pack_values(&job.table, 1, job.row_len);
        const size_t width = (size_t)n * gb > 16 ? 16 : (size_t)n * gb;
        const uint32_t words = (uint32_t)(job.row_len * gb / width);
        const unsigned blocks = (unsigned)device_sm_count() * 8;
        unsigned char *base = static_cast<unsigned char *>(job.table.base);
        const size_t stride = job.table.stride * gb;
        if (width == 16) zero_rows_kernel<uint4><<<blocks, 256, 0, stream>>>(base, stride, job.vocab, words);
        else if (width == 8) zero_rows_kernel<uint2><<<blocks, 256, 0, stream>>>(base, stride, job.vocab, words);
        else if (width == 4) zero_rows_kernel<uint32_t><<<blocks, 256, 0, stream>>>(base, stride, job.vocab, words);
        else zero_rows_kernel<uint16_t><<<blocks, 256, 0, stream>>>(base, stride, job.vocab, words);
        ++*launches;
        timing_mark(stream);
    }
    if (job.n == 0 || job.vocab == 0 || job.row_len == 0) return cudaGetLastError();

    RadixJob r;
    r.kind = KIND_U32;
    r.key_bytes = 4;
    r.val_bytes = 4;
    r.keys_in = t + lay.keys;
    r.keys_out = t + lay.keys_sorted;
    r.keys_alt = t + lay.keys_alt;
    r.vals_in = t + lay.vals;
    r.vals_out = t + lay.vals_sorted;
    r.vals_alt = t + lay.vals_alt;
    r.n = job.n;
    r.begin_bit = 0;
    r.end_bit = 1;
    while ((job.vocab >> r.end_bit) != 0) ++r.end_bit;  // the keys are 0 .. vocab
    r.num_passes = (r.end_bit + 7) / 8;
    r.descending = false;
    r.in_place = false;
    r.hdr = reinterpret_cast<Header *>(t);
    r.hist = reinterpret_cast<uint32_t *>(t + lay.hist);
    r.digit_base = reinterpret_cast<uint32_t *>(t + lay.base);
    r.status = t + lay.status;
    r.wide_status = job.n >= WIDE_STATUS_MIN_KEYS;
    r.num_tiles = lay.tiles;
    debug_fault_settings(&r.fault_pass, &r.fault_tile, &r.spin_limit);
    embedding_keys_kernel<<<(unsigned)((job.n + 255) / 256), 256, 0, stream>>>(
        job.ids, job.id_bytes, job.n, job.first_id, job.padding_id, (uint32_t)job.vocab,
        reinterpret_cast<uint32_t *>(t + lay.keys), reinterpret_cast<uint32_t *>(t + lay.vals));
    ++*launches;
    timing_mark(stream);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_radix_sort(r, stream, launches)) != cudaSuccess) return e;

    GradParams p = {};
    p.keys = reinterpret_cast<uint32_t *>(t + lay.keys_sorted);
    p.vals = reinterpret_cast<uint32_t *>(t + lay.vals_sorted);
    p.n = (uint32_t)job.n;
    p.vocab = (uint32_t)job.vocab;
    p.chunk = chunk_of(job.n, job.row_len);
    p.chunks = lay.chunks;
    p.d_out = static_cast<const unsigned char *>(job.out.base);
    p.grad = static_cast<unsigned char *>(job.table.base);
    p.d_out_stride = job.out.stride * db;
    p.grad_stride = job.table.stride * gb;
    p.row_len = (uint32_t)job.row_len;
    p.scale = job.scale;
    p.accumulate = job.accumulate ? 1 : 0;
    p.partial = reinterpret_cast<float *>(t + lay.partial);
    p.crossing = reinterpret_cast<uint32_t *>(t + lay.crossing);
    p.crossings = reinterpret_cast<uint32_t *>(t + lay.crossings);
    const Rows rows[2] = {job.out, job.table};
    const int n = pack_values(rows, 2, job.row_len);
    if (job.out.type == ROW_F32) return launch_sums_by_grad<float>(p, job.table.type, n, stream, launches);
    if (job.out.type == ROW_F16) return launch_sums_by_grad<__half>(p, job.table.type, n, stream, launches);
    return launch_sums_by_grad<__nv_bfloat16>(p, job.table.type, n, stream, launches);
}

}  // namespace gbs
