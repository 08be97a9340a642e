// Embedding rows looked up by token id, and the table's gradient.
//
//   lookup    out[i] = scale * table[ids[i] - first_id], zeros where the id
//             is outside the table (a shard of a vocabulary)
//   gradient  grad[v] (+)= scale * sum of d_out[i] over ids[i] - first_id = v
//
// The gradient takes the ids in their stable order (id_order.cu), so that each
// table row's terms are neighbours, in the order of i.  The sorted positions
// are cut into chunks; a CTA sums the runs of equal ids of its chunk in 32
// bits.  A run inside one chunk goes to the table at once; a long one that is
// cut leaves 32-bit partial sums, which a second kernel adds in the order of
// the chunks.  No atomics touch a sum, so equal calls give equal bits.  Both
// directions are bound by bytes: one addition per value read.
#include "rows.cuh"

namespace gbs {
namespace {

constexpr int ROW_THREADS = 256;

struct LookupParams {
    const void *ids;
    int id_bytes;
    int64_t first;
    uint64_t n, inside;  // inside: ids_from(first, vocab)
    const unsigned char *table;
    unsigned char *out;
    size_t table_stride, out_stride;  // bytes
    uint32_t row_len, segs, steps, log_lanes, packs;
    float scale;
};

// A warp takes a segment of p.steps * 32 packs of one id's row at a time, its
// id fetched one segment ahead, so that a row's loads wait for no index; all
// loads of a segment are in flight together.  Fewer warps with more in flight
// each are faster: 131072 rows of 4 KB, 8 packs a lane and 2 CTAs an SM 95 us;
// 8 and 3 105; 4 and 4 99; 4 and 6 132.
constexpr int LOOKUP_PACKS = 8, LOOKUP_CTAS = 2;

template <typename T, bool ODD> __global__ void __launch_bounds__(ROW_THREADS, LOOKUP_CTAS) embedding_lookup_kernel(const LookupParams p) {
    constexpr int N = 16 / (int)sizeof(T);
    const uint32_t lane = threadIdx.x & 31;
    __shared__ __align__(16) unsigned char stage[ODD ? ROW_THREADS / 32 : 1][ODD ? LOOKUP_PACKS * 512 + PART_PAD : 16];
    unsigned char *st = stage[ODD ? threadIdx.x >> 5 : 0];
    const uint64_t units = p.n * p.segs, stride = (uint64_t)gridDim.x * (ROW_THREADS / 32);
    uint64_t u = (uint64_t)blockIdx.x * (ROW_THREADS / 32) + (threadIdx.x >> 5);
    wait_for_earlier();
    int32_t next = u < units ? id_index(p.ids, p.id_bytes, u / p.segs, p.first, p.inside) : -1;
    for (; u < units; u += stride) {
        const int32_t at = next;
        if (u + stride < units) next = id_index(p.ids, p.id_bytes, (u + stride) / p.segs, p.first, p.inside);
        const uint32_t c = ((uint32_t)(u % p.segs) * p.steps * 32 + lane) * N;
        const T *src = reinterpret_cast<const T *>(p.table + (size_t)(at < 0 ? 0 : at) * p.table_stride);
        T *dst = reinterpret_cast<T *>(p.out + u / p.segs * p.out_stride);
        Pack<T, N> v[LOOKUP_PACKS];
#pragma unroll
        for (int j = 0; j < LOOKUP_PACKS; ++j) v[j] = load_row<ODD>(src, c + 32 * N * j, p.row_len, at >= 0 && j < (int)p.steps);
        if (p.scale != 1.0f && at >= 0) {
#pragma unroll
            for (int j = 0; j < LOOKUP_PACKS; ++j)
#pragma unroll
                for (int k = 0; k < N; ++k) v[j].v[k] = from_f32<T>(p.scale * to_f32(v[j].v[k]));
        }
#pragma unroll
        for (int j = 0; j < LOOKUP_PACKS; ++j) put_pack<ODD>(dst, c + 32 * N * j, p.row_len, v[j], j < (int)p.steps, st, 32 * j + lane);
        if (ODD) {
            const uint32_t c0 = c - lane * N;
            __syncwarp();
            write_part(reinterpret_cast<unsigned char *>(dst + c0), st, 0, part_bytes<T>(c0, p.steps * 32 * N, p.row_len), lane, 32);
            __syncwarp();
        }
    }
}

// The same for rows of at most LOOKUP_SHORT packs: a warp's turn is as many
// ids as LOOKUP_PACKS packs a lane leave room for, p.steps of each, with
// 2^p.log_lanes lanes to a row; lane l holds the turn's l-th id.  120000 rows of 31
// packs: 21 us, a warp per row 59; of 96 63 against 67, of 128 75 against 73 (64
// against 69 in f32).  Rows at any place, 257 bf16 values: 53 against 106.
constexpr uint32_t LOOKUP_SHORT = 128, LOOKUP_SHORT_ODD = 64;
template <typename T, bool ODD> __global__ void __launch_bounds__(ROW_THREADS, LOOKUP_CTAS) embedding_lookup_short_kernel(const LookupParams p) {
    constexpr int U = LOOKUP_PACKS, N = 16 / (int)sizeof(T);
    const uint32_t lane = threadIdx.x & 31, lanes = 1u << p.log_lanes, per_warp = 32 >> p.log_lanes, which = lane >> p.log_lanes;
    const uint32_t log_steps = __ffs(p.steps) - 1, turn = (p.packs >> log_steps) * per_warp;  // ids of a turn, at most 32
    constexpr uint32_t STAGE = U * 512 + U * (32 >> ODD_LOG_LANES) * PART_PAD;
    __shared__ __align__(16) unsigned char stage[ODD ? ROW_THREADS / 32 * STAGE : 16];
    unsigned char *st = stage + (ODD ? (threadIdx.x >> 5) * STAGE : 0);
    const uint32_t part = p.steps * lanes * 16 + PART_PAD;
    const uint64_t units = (p.n + turn - 1) / turn, stride = (uint64_t)gridDim.x * (ROW_THREADS / 32);
    uint64_t u = (uint64_t)blockIdx.x * (ROW_THREADS / 32) + (threadIdx.x >> 5);
    wait_for_earlier();
    int32_t next = -1;
    if (lane < turn && u * turn + lane < p.n) next = id_index(p.ids, p.id_bytes, u * turn + lane, p.first, p.inside);
    for (; u < units; u += stride) {
        const int32_t now = next;
        const uint64_t i0 = u * turn, ahead = (u + stride) * turn + lane;
        if (lane < turn && ahead < p.n) next = id_index(p.ids, p.id_bytes, ahead, p.first, p.inside);
        const uint32_t c0 = lane & (lanes - 1);
        int32_t at[U];
        Pack<T, N> v[U];
#pragma unroll
        for (int j = 0; j < U; ++j) at[j] = __shfl_sync(~0u, now, ((j >> log_steps) * per_warp + which) & 31);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t c = (c0 + (j & (p.steps - 1)) * lanes) * N, i = (j >> log_steps) * per_warp + which;
            v[j] = load_row<ODD>(reinterpret_cast<const T *>(p.table + (size_t)(at[j] < 0 ? 0 : at[j]) * p.table_stride), c, p.row_len,
                                 at[j] >= 0 && j < (int)p.packs && i0 + i < p.n);
        }
        if (p.scale != 1.0f) {
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int k = 0; k < N; ++k) v[j].v[k] = at[j] < 0 ? T{} : from_f32<T>(p.scale * to_f32(v[j].v[k]));
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t c = (c0 + (j & (p.steps - 1)) * lanes) * N, i = (j >> log_steps) * per_warp + which;
            const bool on = j < (int)p.packs && i0 + i < p.n;
            put_pack<ODD>(reinterpret_cast<T *>(p.out + (on ? i0 + i : 0) * p.out_stride), c, p.row_len, v[j], on, st + i * part,
                          (j & (p.steps - 1)) * lanes + c0);
        }
        if (ODD) {
            __syncwarp();
#pragma unroll 1
            for (uint32_t i = which; i < turn && i0 + i < p.n; i += per_warp)
                write_part(p.out + (i0 + i) * p.out_stride, st + i * part, 0, p.row_len * (uint32_t)sizeof(T), c0, lanes);
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------

struct GradParams {
    const uint32_t *keys, *vals;  // sorted
    uint32_t n, vocab, chunk, chunks;
    const unsigned char *d_out;
    unsigned char *grad;
    size_t d_out_stride, grad_stride;  // bytes
    uint32_t row_len;
    float scale;
    int accumulate;
    uint32_t stages;       // of the ring of rows in flight
    uint32_t lanes;        // that share a short row
    float *partial;        // [2 * chunks][row_len]: a chunk's run from the chunk before, its run into the next
    uint32_t spins;        // tries of a wait of the ring before it gives up
    uint32_t fault_chunk;  // test hook: this chunk's second row is never copied (~0: off)
    uint4 *crossing;       // {first chunk, last chunk, table row} of the runs that are cut, in any order
    uint32_t *crossings;   // how many
    Header *hdr;
};

constexpr uint32_t CHUNK_MOST = 64;

// The positions of one chunk.  A run of equal keys that goes on for at most a
// chunk's length after the border between two chunks belongs to the chunk
// before it, so that only long runs are cut.
struct Chunk {
    uint32_t keys[2 * CHUNK_MOST + 2];  // of the positions from the border's neighbour before it on
    uint32_t vals[2 * CHUNK_MOST];      // from the border on
    uint32_t border[2];
};
// key[1 + j] and val[j] of the chunk's j-th position, key[0] and key[len + 1] of its neighbours
struct Positions {
    const uint32_t *key, *val;
    uint32_t len;
};

// First position from lo on whose sorted key is above k, or n: the warp tries
// 32 places at a time.
__device__ __forceinline__ uint32_t warp_upper_bound(const uint32_t *keys, uint32_t lo, uint32_t n, int64_t k) {
    uint32_t hi = n;
    while (lo < hi) {
        const uint32_t step = (hi - lo + 31) / 32;
        const uint64_t at = (uint64_t)lo + (threadIdx.x & 31) * (uint64_t)step;
        const uint32_t below = __popc(__ballot_sync(~0u, at < hi && (int64_t)keys[at < hi ? at : lo] <= k));
        if (below == 0) break;
        const uint64_t next = (uint64_t)lo + (uint64_t)below * step;
        lo += (below - 1) * step + 1;
        if (next < hi) hi = (uint32_t)next;
    }
    return lo;
}

// The last chunk that begins inside the run that ends before run_end and is
// cut at `border` (so that it goes on there for more than a chunk).
__device__ __forceinline__ uint32_t last_cut(uint32_t run_end, uint32_t border, uint32_t chunk) {
    return max(run_end - 1, border + chunk) / chunk - 1;
}

// Loads the chunk; every thread of the CTA takes part.  A position that adds
// nothing has the key `vocab`, a neighbour that does not exist vocab + 1.
__device__ __forceinline__ Positions load_chunk(const GradParams &p, Chunk &s, uint32_t c) {
    const uint32_t b = c * p.chunk, C = p.chunk, lane = threadIdx.x & 31;
    for (uint32_t j = threadIdx.x; j < 2 * C + 2; j += blockDim.x) {
        const int64_t at = (int64_t)b + j - 1;
        uint32_t k = at >= 0 && at < p.n ? min(p.keys[at], p.vocab) : p.vocab + 1;
        if (j >= 1 && j <= 2 * C && at < p.n) {
            const uint32_t v = p.vals[at];
            s.vals[j - 1] = v;
            if (v >= p.n) k = p.vocab;  // a sort that timed out (the header says so) leaves any values: none is followed
        }
        s.keys[j] = k;
    }
    __syncthreads();
    // where the runs across the borders b and b + C end, counted from the border; 0 where they are cut
    for (uint32_t side = threadIdx.x >> 5; side < 2; side += blockDim.x >> 5) {
        const uint32_t before = s.keys[side * C];
        uint32_t ends = 0;
        for (uint32_t j0 = 0; j0 <= C; j0 += 32) {
            const uint32_t differs = __ballot_sync(~0u, j0 + lane <= C && s.keys[side * C + 1 + min(j0 + lane, C)] != before);
            if (differs) {
                ends = j0 + __ffs(differs) - 1;
                break;
            }
        }
        if (lane == 0) s.border[side] = ends;
    }
    __syncthreads();
    const uint32_t begin = min(b + s.border[0], p.n), end = max(begin, (uint32_t)min((uint64_t)b + C + s.border[1], (uint64_t)p.n)), len = end - begin;
    const Positions at = {s.keys + (begin - b), s.vals + (begin - b), len};
    if (len && blockIdx.y == 0 && threadIdx.x < 32) {
        const uint32_t last = at.key[len];
        if (last < p.vocab && at.key[len + 1] == last && !(at.key[0] == last && at.key[1] == last)) {
            // the last chunk that this run is cut into: it goes on for more than a chunk after that border
            const uint32_t run_end = warp_upper_bound(p.keys, b + C, p.n, last);
            if (threadIdx.x == 0) p.crossing[atomicAdd(p.crossings, 1u)] = make_uint4(c, last_cut(run_end, b + C, C), last, 0);
        }
    }
    return at;
}

template <typename G, int N> __device__ __forceinline__ void to_table(G *dst, const float *acc, float scale, int accumulate,
                                                                      const Pack<G, N> &old) {
    Pack<G, N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.v[i] = from_f32<G>(accumulate ? fmaf(scale, acc[i], to_f32(old.v[i])) : scale * acc[i]);
    store_pack(dst, o);
}
template <int N> __device__ __forceinline__ void to_partial(const GradParams &p, size_t slot, uint32_t c, const float *acc) {
    Pack<float, N> sum;
#pragma unroll
    for (int i = 0; i < N; ++i) sum.v[i] = acc[i];
    store_pack(p.partial + slot * p.row_len + c, sum);
}

// Zeroes the rows of the table that no id names, FILL_ROWS rows per CTA: few
// enough that the last CTAs do not write alone.  8192 ids, 50257 rows of 4 KB, with
// the order and the sums: 8 rows 61.6 us, 16 54.1, 32 53.8, 64 55.7, 128 61.7.
constexpr uint32_t FILL_ROWS = 32;
__device__ void fill_rows(const GradParams &p, uint32_t block, uint32_t byte0, uint32_t bytes) {
    __shared__ uint32_t named[FILL_ROWS / 32], range[2];
    const uint64_t v0 = (uint64_t)block * FILL_ROWS;
    const uint32_t rows = (uint32_t)min((uint64_t)FILL_ROWS, p.vocab - v0);
    if (threadIdx.x < FILL_ROWS / 32) named[threadIdx.x] = 0;
    if (threadIdx.x < 32) {  // the positions of the keys v0 .. v0 + rows - 1
        const uint32_t a = warp_upper_bound(p.keys, 0, p.n, (int64_t)v0 - 1);
        const uint32_t b = warp_upper_bound(p.keys, a, p.n, (int64_t)(v0 + rows) - 1);
        if (threadIdx.x == 0) {
            range[0] = a;
            range[1] = b;
        }
    }
    __syncthreads();
    for (uint32_t j = range[0] + threadIdx.x; j < range[1]; j += blockDim.x) {
        const uint64_t r = p.keys[j] - v0;
        if (r < rows && (j == range[0] || p.keys[j - 1] != p.keys[j])) atomicOr(&named[r / 32], 1u << (r % 32));
    }
    __syncthreads();
    for (uint32_t r = threadIdx.x >> 5; r < rows; r += blockDim.x >> 5) {
        if ((named[r / 32] >> (r % 32)) & 1u) continue;
        zero_bytes(p.grad + (v0 + r) * p.grad_stride + byte0, bytes);
    }
}

// A CTA sums one chunk of sorted positions, a pack of N columns per thread,
// for rows that are not multiples of 16 bytes at multiples of 16 bytes.
template <typename T, typename G, int N> __global__ void __launch_bounds__(ROW_THREADS) embedding_sum_kernel(const GradParams p) {
    __shared__ Chunk s;
    wait_for_earlier();
    if (blockIdx.x >= p.chunks) {
        const uint32_t c0 = blockIdx.y * blockDim.x * N;
        fill_rows(p, blockIdx.x - p.chunks, c0 * (uint32_t)sizeof(G), min(blockDim.x * N, p.row_len - c0) * (uint32_t)sizeof(G));
        return;
    }
    const Positions at = load_chunk(p, s, blockIdx.x);
    const uint32_t len = at.len;
    const uint32_t c = (blockIdx.y * blockDim.x + threadIdx.x) * N;
    if (c >= p.row_len) return;
    float acc[N] = {};
    constexpr uint32_t U = 4;
    bool from_before = at.key[0] == at.key[1];
    for (uint32_t j0 = 0; j0 < len; j0 += U) {
        Pack<T, N> v[U];
#pragma unroll
        for (uint32_t j = 0; j < U; ++j) {
            const bool on = j0 + j < len && at.key[1 + j0 + j] < p.vocab;
            v[j] = load_pack_if<T, N>(reinterpret_cast<const T *>(p.d_out + (on ? at.val[j0 + j] : 0) * p.d_out_stride) + c, on);
        }
#pragma unroll
        for (uint32_t j = 0; j < U; ++j) {
            if (j0 + j >= len || at.key[1 + j0 + j] >= p.vocab) break;
            const uint32_t k = at.key[1 + j0 + j];
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] += to_f32(v[j].v[i]);
            const bool ends = at.key[2 + j0 + j] != k;
            if (ends && !from_before) {
                G *dst = reinterpret_cast<G *>(p.grad + k * p.grad_stride) + c;
                Pack<G, N> old = Pack<G, N>{};
                if (p.accumulate) old = load_pack<G, N>(dst);
                to_table<G, N>(dst, acc, p.scale, p.accumulate, old);
            } else if (ends || j0 + j + 1 == len) {
                to_partial<N>(p, 2 * (size_t)blockIdx.x + (from_before ? 0 : 1), c, acc);
            }
            if (ends) {
                from_before = false;
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] = 0.0f;
            }
        }
    }
}

// The same for rows of whole 16-byte units: the last warp keeps a ring of
// rows in flight by bulk copies (the terms, and the table's row where a run
// ends in it), the others add them up from shared memory, a pack of N columns
// per thread.  A gather of rows by index has one dependent address per row
// and little arithmetic; what bounds it is how many bytes an SM has in
// flight, which the ring sets without registers.  131072 terms of 8 KB into
// 32-bit rows of 16 KB, 2.1 GB: 332 us, 6.5 TB/s, with 4 stages (192 bytes an
// adder), for 256 adders as for 128; 6 stages 336, 8 stages 391 and 395: more
// CTAs with less in flight each are faster.
constexpr int RING_THREADS = 256;     // most threads that add
constexpr uint32_t RING_BYTES = 192;  // of shared memory per thread that adds
constexpr uint32_t RING_STAGES = RING_BYTES / 16;
constexpr uint32_t RING_SPINS = 1u << 20;

__device__ __forceinline__ bool ring_wait(uint64_t *bar, uint32_t parity, uint32_t tries) {
    while (!mbar_try_wait(bar, parity))
        if (--tries == 0) return false;
    return true;
}

// A wait that runs out ends its warp's part: nothing is read from a stage whose
// copy has not come, nothing stored after it, and no stage is given back, so that
// the copying warp's own wait runs out in turn.  That warp stays until every copy
// that it has asked for has come: the shared memory is another CTA's after this
// one.
template <typename T, typename G> __global__ void __launch_bounds__(RING_THREADS + 32) embedding_ring_kernel(const GradParams p) {
    constexpr int N = 16 / (int)sizeof(T);
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ Chunk s;
    __shared__ alignas(8) uint64_t full[RING_STAGES], empty[RING_STAGES];
    const uint32_t adders = blockDim.x - 32, lane = threadIdx.x & 31;
    const uint32_t c0 = blockIdx.y * adders * N, cols = min(adders * N, p.row_len - c0);
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < p.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], adders / 32);
        }
        fence_mbar_init();
    }
    wait_for_earlier();
    if (blockIdx.x >= p.chunks) {
        fill_rows(p, blockIdx.x - p.chunks, c0 * (uint32_t)sizeof(G), cols * (uint32_t)sizeof(G));
        return;
    }
    const Positions pos = load_chunk(p, s, blockIdx.x);  // also makes the barriers visible
    const uint32_t len = pos.len;
    const uint32_t term_bytes = adders * 16, stage_bytes = term_bytes + (p.accumulate ? adders * N * (uint32_t)sizeof(G) : 0);
    bool late = false;
    const bool cut = pos.key[0] == pos.key[1];  // the first run began in a chunk before
    if (threadIdx.x >= adders) {
        if (lane != 0) return;
        bool from_before = cut;
        const uint32_t withheld = blockIdx.x == p.fault_chunk ? 1 : ~0u;
        uint32_t j = 0;
        for (; j < len; ++j) {
            const uint32_t k = pos.key[1 + j], st = j % p.stages;
            if (k >= p.vocab) break;
            if (j >= p.stages && !ring_wait(&empty[st], (j / p.stages - 1) & 1, p.spins)) {
                late = true;
                break;
            }
            const bool ends = pos.key[2 + j] != k, old = p.accumulate && ends && !from_before;
            if (ends) from_before = false;
            if (j == withheld) continue;
            const uint32_t term = cols * (uint32_t)sizeof(T), row = cols * (uint32_t)sizeof(G);
            mbar_arrive_expect_tx(&full[st], term + (old ? row : 0));
            bulk_g2s(ring + st * stage_bytes, p.d_out + pos.val[j] * p.d_out_stride + c0 * sizeof(T), term, &full[st]);
            if (old) bulk_g2s(ring + st * stage_bytes + term_bytes, p.grad + k * p.grad_stride + c0 * sizeof(G), row, &full[st]);
        }
        for (uint32_t i = j > p.stages ? j - p.stages : 0; i < j; ++i)
            if (i != withheld) late |= !ring_wait(&full[i % p.stages], (i / p.stages) & 1, RING_SPINS);
        if (late) record_error(p.hdr, ERR_COPY_TIMEOUT, blockIdx.x);
        return;
    }
    const uint32_t c = c0 + threadIdx.x * N;
    const bool inside = c < p.row_len;
    float acc[N] = {};
    bool from_before = cut;
    for (uint32_t j = 0; j < len; ++j) {
        const uint32_t k = pos.key[1 + j], st = j % p.stages;
        if (k >= p.vocab) break;
        late = __any_sync(~0u, !ring_wait(&full[st], (j / p.stages) & 1, p.spins));
        if (late) break;
        const unsigned char *at = ring + st * stage_bytes;
        const Pack<T, N> v = *reinterpret_cast<const Pack<T, N> *>(at + threadIdx.x * 16);
        const bool ends = pos.key[2 + j] != k, direct = ends && !from_before;
        Pack<G, N> old = Pack<G, N>{};
        if (direct && p.accumulate) old = *reinterpret_cast<const Pack<G, N> *>(at + term_bytes + threadIdx.x * N * sizeof(G));
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += to_f32(v.v[i]);
        if (inside) {
            if (direct) to_table<G, N>(reinterpret_cast<G *>(p.grad + k * p.grad_stride) + c, acc, p.scale, p.accumulate, old);
            else if (ends || j + 1 == len) to_partial<N>(p, 2 * (size_t)blockIdx.x + (from_before ? 0 : 1), c, acc);
        }
        if (ends) {
            from_before = false;
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = 0.0f;
        }
    }
    if (late && lane == 0) record_error(p.hdr, ERR_COPY_TIMEOUT, blockIdx.x);
}

// The same for rows of fewer than 32 packs of 16 bytes: p.lanes lanes take a
// chunk, and a warp takes 32 / p.lanes neighbouring chunks, whose positions it
// loads at once.
constexpr int SHORT_THREADS = 128;
constexpr uint32_t SHORT_CHUNK_MOST = 32;
template <typename T, typename G> __global__ void __launch_bounds__(SHORT_THREADS) embedding_short_kernel(const GradParams p) {
    constexpr int N = 16 / (int)sizeof(T);
    constexpr uint32_t SPAN = 17 * SHORT_CHUNK_MOST + 2;
    // keys[1 + j], vals[j]: position j of the warp's span; a position that adds nothing has the key `vocab`, one that
    // does not exist vocab + 1
    __shared__ uint32_t all_keys[SHORT_THREADS / 32][SPAN], all_vals[SHORT_THREADS / 32][SPAN];
    const uint32_t lane = threadIdx.x & 31, per_warp = 32 / p.lanes, sum_blocks = (p.chunks + SHORT_THREADS / p.lanes - 1) / (SHORT_THREADS / p.lanes);
    wait_for_earlier();
    if (blockIdx.x >= sum_blocks) {
        fill_rows(p, blockIdx.x - sum_blocks, 0, p.row_len * (uint32_t)sizeof(G));
        return;
    }
    uint32_t *const keys = all_keys[threadIdx.x >> 5], *const vals = all_vals[threadIdx.x >> 5];
    const uint32_t q0 = (blockIdx.x * (SHORT_THREADS / 32) + (threadIdx.x >> 5)) * per_warp, C = p.chunk, span = (per_warp + 1) * C;
    const int64_t b = (int64_t)q0 * C;
#pragma unroll 4
    for (uint32_t j = lane; j < span + 2; j += 32) {
        const int64_t at = b + j - 1;
        uint32_t k = p.vocab + 1, v = 0;
        if (at >= 0 && at < p.n) {
            k = min(p.keys[at], p.vocab);
            v = p.vals[at];
            if (v >= p.n) k = p.vocab;  // a sort that timed out leaves any values: none is followed outside d_out
        }
        keys[j] = k;
        if (j >= 1) vals[j - 1] = v;
    }
    __syncwarp();
    // the chunks' borders, a lane each (17 at most): after the run that crosses it, if that ends within a chunk's length
    const uint32_t here = min(lane, per_warp) * C, most = (uint32_t)min((int64_t)span, max((int64_t)p.n - b, (int64_t)0));
    uint32_t more = 0;
    while (more <= C && keys[here + more + 1] == keys[here]) ++more;
    const uint32_t border = min(more <= C ? here + more : here, most);
    const uint32_t which = lane / p.lanes, col = lane % p.lanes * N, c = q0 + which;
    const uint32_t begin = __shfl_sync(~0u, border, which), end = max(begin, __shfl_sync(~0u, border, which + 1));
    bool from_before = begin < end && keys[begin + 1] == keys[begin];
    // the chunk's last run goes on in the next and begins here: list it, one chunk after another
    const bool starts = begin < end && keys[end] < p.vocab && keys[end + 1] == keys[end] && !(from_before && keys[begin + 1] == keys[end]);
    uint32_t todo = __ballot_sync(~0u, starts && lane % p.lanes == 0);
    while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const uint32_t e = __shfl_sync(~0u, end, src), chunk = __shfl_sync(~0u, c, src), k = keys[e];
        const uint32_t run_end = warp_upper_bound(p.keys, (uint32_t)(b + e), p.n, k);
        if (lane == 0) p.crossing[atomicAdd(p.crossings, 1u)] = make_uint4(chunk, last_cut(run_end, (chunk + 1) * C, C), k, 0);
    }
    if (col >= p.row_len) return;
    float acc[N] = {};
    constexpr uint32_t U = 4;
    for (uint32_t j0 = begin; j0 < end; j0 += U) {
        uint32_t k[U + 1], val[U];
#pragma unroll
        for (uint32_t j = 0; j <= U; ++j) k[j] = keys[min(1 + j0 + j, span + 1)];
#pragma unroll
        for (uint32_t j = 0; j < U; ++j) val[j] = vals[min(j0 + j, span)];
        Pack<T, N> v[U];
        Pack<G, N> old[U];
#pragma unroll
        for (uint32_t j = 0; j < U; ++j) {
            const bool on = j0 + j < end && k[j] < p.vocab;
            v[j] = load_pack_if<T, N>(reinterpret_cast<const T *>(p.d_out + (on ? val[j] : 0) * p.d_out_stride) + col, on);
            old[j] = load_own_if<G, N>(reinterpret_cast<const G *>(p.grad + (on ? k[j] : 0) * p.grad_stride) + col,
                                       on && p.accumulate && k[j + 1] != k[j]);
        }
#pragma unroll
        for (uint32_t j = 0; j < U; ++j) {
            if (j0 + j >= end || k[j] >= p.vocab) break;
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] += to_f32(v[j].v[i]);
            const bool ends = k[j + 1] != k[j];
            if (ends && !from_before)
                to_table<G, N>(reinterpret_cast<G *>(p.grad + k[j] * p.grad_stride) + col, acc, p.scale, p.accumulate, old[j]);
            else if (ends || j0 + j + 1 == end)
                to_partial<N>(p, 2 * (size_t)c + (from_before ? 0 : 1), col, acc);
            if (ends) {
                from_before = false;
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] = 0.0f;
            }
        }
    }
}

// Adds the partial sums of the runs that are cut: an item is one such run and
// 32 packs of columns.  The warps share the run's chunks, each in order, and
// the CTA adds the warps' sums in order.  Bound by the latency of an item (its
// entry, its sums, the table's row): the cut runs of 131072 ids x 4096 columns
// take 16 us.
constexpr int JOIN_THREADS = 512;
template <typename G, int N> __global__ void __launch_bounds__(JOIN_THREADS) embedding_join_kernel(const GradParams p) {
    constexpr int WARPS = JOIN_THREADS / 32;
    __shared__ float sums[WARPS][32 * N];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t blocks = (p.row_len + 32 * N - 1) / (32 * N);
    wait_for_earlier();
    const uint64_t items = (uint64_t)*p.crossings * blocks;
    for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const uint4 run = p.crossing[it / blocks];
        const uint32_t c = (uint32_t)(it % blocks) * 32 * N + lane * N;
        G *dst = reinterpret_cast<G *>(p.grad + run.z * p.grad_stride) + c;
        Pack<G, N> old = Pack<G, N>{};
        if (warp == 0 && c < p.row_len && p.accumulate) old = load_pack<G, N>(dst);
        float acc[N] = {};
        if (c < p.row_len) {
#pragma unroll 4
            for (uint32_t q = run.x + warp; q <= run.y; q += WARPS) {
                const Pack<float, N> sum = load_pack<float, N>(p.partial + (2 * (size_t)q + (q == run.x ? 1 : 0)) * p.row_len + c);
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] += sum.v[i];
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) sums[warp][32 * i + lane] = acc[i];
        __syncthreads();
        if (warp == 0 && c < p.row_len) {
            const uint32_t used = min((uint32_t)WARPS, run.y - run.x + 1);
            for (uint32_t w = 1; w < used; ++w)
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] += sums[w][32 * i + lane];
            to_table<G, N>(dst, acc, p.scale, p.accumulate, old);
        }
        __syncthreads();
    }
}

// The whole gradient of a short list in one launch, without a sort: a CTA
// takes FEW_IDS positions, a warp each.  The warp compares its id with all
// others, 32 at a time; where one before it is equal, that one's warp has the
// row, else it lists the equal ones in order.  The CTA's warps then share the
// columns of the lists, or, where a list is long, its parts, which are added in
// order.  That reads every id once per CTA, n^2 / 8 in all, against the launches
// of an order, its sums and their joining (1024 ids x 1024 bf16 values 6.8 us, by
// way of an order 9.6, and one launch on the host instead of three).  What bounds it
// is the chain of
// ids, ballots, terms and the table's row.
constexpr uint32_t FEW_MOST = 1024;  // a lane for each 32 positions
constexpr int FEW_IDS = 8, FEW_THREADS = 32 * FEW_IDS;
constexpr uint32_t FEW_LONG = 16;  // a list above this is shared by the warps
struct FewParams {
    const void *ids;
    int id_bytes;
    int64_t first, padding;
    uint32_t inside;       // ids_from(first, vocab)
    uint32_t pack_blocks;  // blocks of 32 packs of columns that make a row
    uint32_t per_cta;      // of them per CTA
    uint32_t id_blocks;    // CTAs that sum; the others zero fill_rows rows each
    uint32_t fill_rows;
};
// The position that a CTA's warp takes.  Frequent ids have their first
// position early in the list: neighbours go to different CTAs.
__device__ __forceinline__ uint32_t few_id(const FewParams &f, uint32_t warp) { return warp * f.id_blocks + blockIdx.x; }

template <typename T, typename G, int N> __global__ void __launch_bounds__(FEW_THREADS) embedding_few_kernel(const GradParams p, const FewParams f) {
    __shared__ uint32_t key[FEW_MOST];
    __shared__ uint16_t list[FEW_IDS][FEW_MOST];
    __shared__ uint32_t count[FEW_IDS];
    __shared__ float sums[FEW_IDS][32 * N];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blocks = (p.n + 31) / 32;
    wait_for_earlier();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) p.hdr->error = 0;  // no wait here can run out
    if (f.id_bytes == 8) load_keys(key, static_cast<const int64_t *>(f.ids), p.n, blocks * 32, f.first, f.padding, f.inside, p.vocab);
    else load_keys(key, static_cast<const int32_t *>(f.ids), p.n, blocks * 32, f.first, f.padding, f.inside, p.vocab);
    __syncthreads();
    const uint32_t b0 = blockIdx.y * f.per_cta, b1 = min(b0 + f.per_cta, f.pack_blocks);
    if (blockIdx.x >= f.id_blocks) {  // rows that no id names
        uint32_t *named = count;
        const uint64_t v0 = ((uint64_t)(blockIdx.x - f.id_blocks) * gridDim.y + blockIdx.y) * f.fill_rows;
        if (v0 >= p.vocab) return;
        const uint32_t rows = (uint32_t)min((uint64_t)f.fill_rows, p.vocab - v0);
        if (threadIdx.x < FILL_ROWS / 32) named[threadIdx.x] = 0;
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < p.n; i += FEW_THREADS)
            if (key[i] - v0 < rows) atomicOr(&named[(key[i] - v0) / 32], 1u << ((key[i] - v0) % 32));
        __syncthreads();
        for (uint32_t r = warp; r < rows; r += FEW_IDS)
            if (!((named[r / 32] >> (r % 32)) & 1u)) zero_bytes(p.grad + (v0 + r) * p.grad_stride, p.row_len * (uint32_t)sizeof(G));
        return;
    }
    {
        const uint32_t i = few_id(f, warp), k = i < p.n ? key[i] : p.vocab;
        uint32_t equal = 0;  // lane b: which of the b-th 32 positions are equal
#pragma unroll 8
        for (uint32_t b = 0; b < blocks; ++b) {
            const uint32_t m = __ballot_sync(~0u, key[32 * b + lane] == k);
            if (lane == b) equal = m;
        }
        const uint32_t earlier = lane < i / 32 ? equal : lane == i / 32 ? equal & ((1u << (i % 32)) - 1) : 0;
        const bool first = !__any_sync(~0u, earlier) && k < p.vocab;
        uint32_t at = __popc(equal), found;
#pragma unroll
        for (int s = 1; s < 32; s *= 2) {
            const uint32_t o = __shfl_up_sync(~0u, at, s);
            if (lane >= (uint32_t)s) at += o;
        }
        found = __shfl_sync(~0u, at, 31);
        at -= __popc(equal);
        for (uint32_t m = first ? equal : 0; m; m &= m - 1) list[warp][at++] = (uint16_t)(32 * lane + __ffs(m) - 1);
        if (lane == 0) count[warp] = first ? found : 0;
    }
    __syncthreads();
    const auto add_up = [&](uint32_t w, uint32_t q0, uint32_t q1, uint32_t c, float *acc) {
        constexpr uint32_t U = 8;
        for (uint32_t q = q0; q < q1; q += U) {
            Pack<T, N> v[U];
#pragma unroll
            for (uint32_t j = 0; j < U; ++j) {
                const bool on = q + j < q1;
                v[j] = load_pack_if<T, N>(reinterpret_cast<const T *>(p.d_out + (on ? list[w][q + j] : 0) * p.d_out_stride) + c, on && c < p.row_len);
            }
#pragma unroll
            for (uint32_t j = 0; j < U; ++j)
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] += to_f32(v[j].v[i]);
        }
    };
    const auto row_of = [&](uint32_t w) { return reinterpret_cast<G *>(p.grad + key[few_id(f, w)] * p.grad_stride); };
    for (uint32_t it = warp; it < FEW_IDS * (b1 - b0); it += FEW_IDS) {
        // a warp takes another list for each block of columns, so that one long list does not stay with it
        const uint32_t w = (warp + it / FEW_IDS) % FEW_IDS, c = ((b0 + it / FEW_IDS) * 32 + lane) * N, most = count[w];
        if (most == 0 || most > FEW_LONG) continue;
        G *dst = row_of(w) + c;
        const Pack<G, N> old = load_own_if<G, N>(dst, p.accumulate && c < p.row_len);
        float acc[N] = {};
        add_up(w, 0, most, c, acc);
        if (c < p.row_len) to_table<G, N>(dst, acc, p.scale, p.accumulate, old);
    }
    for (uint32_t w = 0; w < FEW_IDS; ++w) {
        const uint32_t most = count[w];
        if (most <= FEW_LONG) continue;
        for (uint32_t b = b0; b < b1; ++b) {
            const uint32_t c = (b * 32 + lane) * N;
            G *dst = row_of(w) + c;
            Pack<G, N> old = Pack<G, N>{};
            if (warp == 0) old = load_own_if<G, N>(dst, p.accumulate && c < p.row_len);
            float acc[N] = {};
            add_up(w, most * warp / FEW_IDS, most * (warp + 1) / FEW_IDS, c, acc);
#pragma unroll
            for (int i = 0; i < N; ++i) sums[warp][32 * i + lane] = acc[i];
            __syncthreads();
            if (warp == 0 && c < p.row_len) {
                for (int part = 1; part < FEW_IDS; ++part)
#pragma unroll
                    for (int i = 0; i < N; ++i) acc[i] += sums[part][32 * i + lane];
                to_table<G, N>(dst, acc, p.scale, p.accumulate, old);
            }
            __syncthreads();
        }
    }
}

// Sorted positions of a chunk: long ones for long lists (fewer borders),
// short ones while the chunks would not fill the SMs.  131072 x 4096: with
// 64 positions 332 us, and 16 to join what is cut; with 128 356 and 10, with 32
// 324 and 29.
uint32_t chunk_of(size_t n, size_t row_len) {
    uint32_t chunk = row_len < 256 ? SHORT_CHUNK_MOST : CHUNK_MOST;  // short rows' chunks lie in shared memory together
    const size_t slices = (row_len + 1023) / 1024;
    while (chunk > 8 && n / chunk * slices < 152 * 16) chunk /= 2;  // 16 CTAs for each of 152 SMs
    return chunk;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// The header and the count of cut runs come first: the order's first kernel
// clears both.
struct GradLayout {
    size_t crossings, order, keys, vals, crossing, partial, total;
    uint32_t chunks;
};
GradLayout grad_layout(size_t n, size_t vocab, size_t row_len) {
    GradLayout l;
    const size_t chunk = chunk_of(n, row_len), list = up(sizeof(uint32_t) * n);
    l.chunks = (uint32_t)((n + chunk - 1) / chunk);
    size_t off = sizeof(Header);
    l.crossings = off;
    l.order = off = ID_ORDER_CLEARED;
    l.keys = off += up(id_order_temp_bytes(n, vocab));
    l.vals = off += list;
    l.crossing = off += list;
    l.partial = off += up(sizeof(uint4) * (size_t)l.chunks);
    l.total = off + up(sizeof(float) * 2 * l.chunks * row_len);
    return l;
}

// Whether the short list's kernel takes a call: it compares all ids in every
// CTA.  bf16 rows: 1024 ids x 1024 values 6.8 us, by way of an order 9.6; 512 x
// 4096, 1024 of these pieces, 9.6 against 9.2 with half its host time; 1024 x
// 4096 13.8 against 10.9.  f32 rows: 512 x 2048 8.2 against 8.9, 384 x 4096, 1536
// pieces, 8.2 against 8.9, 512 x 4096 10.2 against 8.9.
bool is_few(size_t n, size_t packs) {
    return n <= FEW_MOST && (n + FEW_IDS - 1) / FEW_IDS * ((packs + 31) / 32) <= 1024;
}

template <typename T, typename G, int N> cudaError_t launch_few(const GradParams &p, FewParams f, cudaStream_t stream, int *launches) {
    const uint32_t sms = (uint32_t)device_sm_count();
    f.id_blocks = (p.n + FEW_IDS - 1) / FEW_IDS;
    f.pack_blocks = (p.row_len / N + 31) / 32;
    f.fill_rows = FILL_ROWS;  // 128 KB, where rows are wide: 200 ids into 5000 rows of 16 KB 20.5 us instead of 35.5
    while (f.fill_rows > 4 && (size_t)f.fill_rows * p.row_len * sizeof(G) > 128 * 1024) f.fill_rows /= 2;
    f.per_cta = 1;  // a CTA compares its ids once for all of its columns
    while (f.per_cta < f.pack_blocks && (uint64_t)f.id_blocks * ((f.pack_blocks + f.per_cta - 1) / f.per_cta) > 8 * sms) f.per_cta *= 2;
    if (f.id_blocks == 0) f.per_cta = f.pack_blocks;  // the rows are only zeroed, whole: no slices of columns
    const uint32_t slices = (f.pack_blocks + f.per_cta - 1) / f.per_cta, rows = slices * f.fill_rows;
    const dim3 grid(f.id_blocks + (p.accumulate ? 0 : (p.vocab + rows - 1) / rows), slices);
    const cudaError_t e = launch_next(embedding_few_kernel<T, G, N>, grid, FEW_THREADS, 0, stream, p, f);
    ++*launches;
    timing_mark(stream);
    return e;
}

template <typename T, typename G, int N> cudaError_t launch_sums(GradParams p, cudaStream_t stream, int *launches) {
    const uint32_t packs = p.row_len / N;
    const bool whole = N * sizeof(T) == 16;  // rows are 16-byte units in both matrices
    const bool brief = whole && packs < 32, ring = whole && !brief;
    // columns in slices of equal length, a warp's 32 packs at least
    const uint32_t most = ring ? RING_THREADS : ROW_THREADS, slices = (packs + most - 1) / most;
    const uint32_t threads = ((packs + slices - 1) / slices + 31) / 32 * 32;
    const uint32_t fills = p.accumulate ? 0 : (p.vocab + FILL_ROWS - 1) / FILL_ROWS;
    cudaError_t e = cudaSuccess;
    const dim3 grid(p.chunks + fills, (packs + threads - 1) / threads);
    if constexpr (N * sizeof(T) == 16) {
        if (ring) {
            const uint32_t stage = threads * (16 + (p.accumulate ? N * (uint32_t)sizeof(G) : 0));
            p.stages = RING_BYTES * threads / stage;
            static PerDeviceOnce once;
            e = once.run([] {
                return cudaFuncSetAttribute(embedding_ring_kernel<T, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)RING_BYTES * RING_THREADS);
            });
            if (e != cudaSuccess) return e;
            e = launch_next(embedding_ring_kernel<T, G>, grid, threads + 32, p.stages * stage, stream, p);
        }
    }
    if constexpr (N * sizeof(T) == 16) {
        if (brief) {
            p.lanes = 2;
            while (p.lanes < packs) p.lanes *= 2;
            const uint32_t per_block = SHORT_THREADS / p.lanes;
            e = launch_next(embedding_short_kernel<T, G>, (p.chunks + per_block - 1) / per_block + fills, SHORT_THREADS, 0, stream, p);
        }
    }
    if constexpr (N * sizeof(T) != 16) e = launch_next(embedding_sum_kernel<T, G, N>, grid, threads, 0, stream, p);
    if (e != cudaSuccess) return e;
    ++*launches;
    timing_mark(stream);
    if (p.chunks > 1) {
        e = launch_next(embedding_join_kernel<G, N>, (unsigned)device_sm_count() * 4, JOIN_THREADS, 0, stream, p);
        ++*launches;
        timing_mark(stream);
    }
    return e;
}

template <typename T, typename G> cudaError_t launch_sums_by_width(const GradParams &p, const FewParams &f, int n, cudaStream_t stream, int *launches) {
    constexpr int FULL = 16 / (int)sizeof(T);
    if (is_few(p.n, p.row_len / (n >= FULL ? FULL : n >= 2 ? 2 : 1))) {
        if (n >= FULL) return launch_few<T, G, FULL>(p, f, stream, launches);
        return n >= 2 ? launch_few<T, G, 2>(p, f, stream, launches) : launch_few<T, G, 1>(p, f, stream, launches);
    }
    if (n >= FULL) return launch_sums<T, G, FULL>(p, stream, launches);
    if (n >= 2) return launch_sums<T, G, 2>(p, stream, launches);
    return launch_sums<T, G, 1>(p, stream, launches);
}

template <typename T> cudaError_t launch_sums_by_grad(const GradParams &p, const FewParams &f, int type, int n, cudaStream_t stream, int *launches) {
    if (type == ROW_F32) return launch_sums_by_width<T, float>(p, f, n, stream, launches);
    return launch_sums_by_width<T, T>(p, f, n, stream, launches);
}

template <typename T, bool ODD> cudaError_t launch_lookup(LookupParams p, cudaStream_t stream) {
    const uint32_t packs = (p.row_len * (uint32_t)sizeof(T) + 15) / 16;
    const unsigned most = (unsigned)device_sm_count() * LOOKUP_CTAS;
    const uint64_t most_warps = 2 * most * (ROW_THREADS / 32);
    if (packs > (ODD ? LOOKUP_SHORT_ODD : LOOKUP_SHORT)) {
        p.steps = LOOKUP_PACKS;  // short segments give every warp work when there are few ids
        while (p.steps > 1 && p.n * ((packs + 32 * p.steps - 1) / (32 * p.steps)) < most_warps) p.steps /= 2;
        p.segs = (packs + 32 * p.steps - 1) / (32 * p.steps);
        p.steps = (packs + 32 * p.segs - 1) / (32 * p.segs);  // segments of equal length
        const uint64_t blocks = (p.n * p.segs + ROW_THREADS / 32 - 1) / (ROW_THREADS / 32);
        return launch_next(embedding_lookup_kernel<T, ODD>, (unsigned)(blocks < most ? blocks : most), ROW_THREADS, 0, stream, p);
    }
    p.log_lanes = ODD ? ODD_LOG_LANES : 0;
    while ((1u << p.log_lanes) < packs && p.log_lanes < 5) ++p.log_lanes;
    p.steps = packs > 64 ? 4 : packs > 32 ? 2 : 1;
    p.packs = LOOKUP_PACKS;
    const uint32_t per_warp = 32 >> p.log_lanes;
    while (p.packs > p.steps && (p.packs / p.steps * per_warp > 32 || p.n / (p.packs / p.steps * per_warp) < most * (ROW_THREADS / 32))) p.packs /= 2;
    const uint32_t turn = p.packs / p.steps * per_warp;
    const uint64_t blocks = ((p.n + turn - 1) / turn + ROW_THREADS / 32 - 1) / (ROW_THREADS / 32);
    return launch_next(embedding_lookup_short_kernel<T, ODD>, (unsigned)(blocks < most ? blocks : most), ROW_THREADS, 0, stream, p);
}

template <typename T> cudaError_t launch_lookup_of(const LookupParams &p, bool any, cudaStream_t stream) {
    return any ? launch_lookup<T, true>(p, stream) : launch_lookup<T, false>(p, stream);
}

}  // namespace

cudaError_t launch_embedding_lookup(const EmbeddingJob &job, cudaStream_t stream, int *launches) {
    LookupParams p = {};
    const size_t b = (size_t)row_bytes(job.table.type);
    p.ids = job.ids;
    p.id_bytes = job.id_bytes;
    p.first = job.first_id;
    p.n = job.n;
    p.inside = ids_from(job.first_id, job.vocab);
    p.table = static_cast<const unsigned char *>(job.table.base);
    p.out = static_cast<unsigned char *>(job.out.base);
    p.table_stride = job.table.stride * b;
    p.out_stride = job.out.stride * b;
    p.row_len = (uint32_t)job.row_len;
    p.scale = job.scale;
    const Rows rows[2] = {job.table, job.out};
    const bool any = !whole_packs(rows, 2, job.row_len);
    const cudaError_t e = job.table.type == ROW_F32   ? launch_lookup_of<float>(p, any, stream)
                          : job.table.type == ROW_F16 ? launch_lookup_of<__half>(p, any, stream)
                                                      : launch_lookup_of<__nv_bfloat16>(p, any, stream);
    ++*launches;
    timing_mark(stream);
    return e;
}

size_t embedding_grad_temp_bytes(size_t n, size_t vocab, size_t row_len) {
    return grad_layout(n, vocab, row_len).total;
}

cudaError_t launch_embedding_grad(const EmbeddingJob &job, cudaStream_t stream, int *launches) {
    const GradLayout lay = grad_layout(job.n, job.vocab, job.row_len);
    unsigned char *t = job.temp;
    const size_t gb = (size_t)row_bytes(job.table.type), db = (size_t)row_bytes(job.out.type);
    Header *hdr = reinterpret_cast<Header *>(t);
    if (job.vocab == 0 || job.row_len == 0 || (job.n == 0 && job.accumulate))
        return cudaMemsetAsync(hdr, 0, sizeof(Header), stream);
    IdOrderJob order = {};
    order.ids = job.ids;
    order.id_bytes = job.id_bytes;
    order.n = job.n;
    order.vocab = job.vocab;
    order.first_id = job.first_id;
    order.padding_id = job.padding_id;
    order.hdr = hdr;
    order.work = t + lay.order;
    order.keys = reinterpret_cast<uint32_t *>(t + lay.keys);
    order.vals = reinterpret_cast<uint32_t *>(t + lay.vals);
    FewParams f = {};
    f.ids = job.ids;
    f.id_bytes = job.id_bytes;
    f.first = job.first_id;
    f.padding = job.padding_id;
    f.inside = (uint32_t)ids_from(job.first_id, job.vocab);
    GradParams p = {};
    p.keys = order.keys;
    p.vals = order.vals;
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
    p.crossing = reinterpret_cast<uint4 *>(t + lay.crossing);
    p.crossings = reinterpret_cast<uint32_t *>(t + lay.crossings);
    p.hdr = hdr;
    debug_ring_settings(&p.fault_chunk, &p.spins);
    if (p.spins == 0) p.spins = RING_SPINS;
    const Rows rows[2] = {job.out, job.table};
    const int n = pack_values(rows, 2, job.row_len), full = 16 / (int)db;
    if (!is_few(job.n, job.row_len / (size_t)(n >= full ? full : n >= 2 ? 2 : 1))) {
        const cudaError_t e = launch_id_order(order, stream, launches);
        if (e != cudaSuccess) return e;
    }
    if (job.out.type == ROW_F32) return launch_sums_by_grad<float>(p, f, job.table.type, n, stream, launches);
    if (job.out.type == ROW_F16) return launch_sums_by_grad<__half>(p, f, job.table.type, n, stream, launches);
    return launch_sums_by_grad<__nv_bfloat16>(p, f, job.table.type, n, stream, launches);
}

}  // namespace gbs
