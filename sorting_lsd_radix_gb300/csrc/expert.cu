// Token rows grouped by expert and back.
//
// A router gives every token t the experts e(t, k), k < top_k.  The slots
// s = t * top_k + k are sorted stably by expert, which is one counting sort:
//   row(s) = offsets[e(s)] + #{s' < s : e(s') = e(s)},
// with offsets the running sum of the experts' counts, each rounded up to
// row_align.  Slots whose expert is not in [first, first + experts) have no
// row.  The rows then move in that order:
//   dispatch / gather  rows[row(t, k)] = x[t], zeros in rows without a slot
//   combine            out[t] = sum_k w[t, k] * rows[row(t, k)]
//   combine's gradient d_rows[row(t, k)] = w[t, k] * d_out[t],
//                      d_w[t, k] = d_out[t] . rows[row(t, k)]
// (gather's gradient is combine without weights.)  All of them are bound by
// the rows' bytes: there are at most three operations per value moved.
#include "rows.cuh"

namespace gbs {
namespace {

constexpr int HERE_THREADS = 512;     // of a CTA that counts every slot
constexpr int TILE_THREADS = 256;     // of one whose counts are made before
constexpr int GROUP_TILES = 8;        // tiles that a CTA counts, one per warp
// Up to this many slots every CTA counts all of them by itself (one launch);
// above, a CTA's warps count a tile each into the work buffer.
// 16384 slots of 128 experts and rows of 2 KB: 13.4 us either way; 32768: 23.7
// counted by every CTA, 21.8 by tiles.
constexpr size_t COUNT_HERE_SLOTS = 16384;
// Slots of such a tile: enough tiles for eight CTAs on each of 152 SMs, and at
// least 32 slots; 4096 above LONG_SLOTS, to bound the work buffer.
constexpr size_t TILE_SLOTS_LEAST = 32, TILE_SLOTS = 256, TILE_SLOTS_LONG = 4096, LONG_SLOTS = (size_t)1 << 22;
// Rows of this many bytes or more move in a launch of their own, whose many
// short CTAs write faster than the tiles' (2.1 GB: 356 us of 379 with the order,
// 394 with the tiles; 134 MB: 27 of 37, 36 with the tiles).
constexpr size_t APART_BYTES = (size_t)512 << 20;
constexpr int SEG_WORDS = 4;  // units of 16 bytes of a row that a lane moves at once
// A warp's shared memory for rows at any place: its lanes' segments and their ends.
constexpr uint32_t MOVE_STAGE = 32 * SEG_WORDS * 16 + (32 >> ODD_LOG_LANES) * PART_PAD;

// How rows move: by words of 16, 8, 4 or 2 bytes, or (ODD_WORD) by aligned words of
// 16 bytes through shared memory, which takes more instructions for a row and
// fewer for a byte: rows that only 2-byte words fit, from ODD_BYTES on (200000
// slots of 739 bf16 values 112 -> 94 us; of 222 36 -> 54).
constexpr int ODD_WORD = 0;
constexpr uint32_t ODD_BYTES = 1024;
constexpr uint32_t unit_bytes(int word) { return word == ODD_WORD ? 16 : (uint32_t)word; }

// Moves a segment of a row to each of its slots' rows: unit c (of a word, or 16
// bytes) on, `lanes` lanes, this one as `sub`.  ODD_WORD: the warp takes part as
// a whole, and st is the lanes' part of shared memory, SEG_WORDS * lanes units
// and two.
template <int WORD, typename RowOf>
__device__ __forceinline__ void move_segment(const unsigned char *src, uint32_t c, uint32_t sub, uint32_t lanes, uint32_t row_bytes, bool on,
                                             uint32_t top_k, RowOf row_of, unsigned char *rows, size_t stride, unsigned char *st) {
    if constexpr (WORD != ODD_WORD) {
        constexpr int N = WORD / 2;
        if (!on) return;
        Pack<uint16_t, N> v[SEG_WORDS];
#pragma unroll
        for (int i = 0; i < SEG_WORDS; ++i)
            v[i] = load_pack_if<uint16_t, N>(reinterpret_cast<const uint16_t *>(src) + (c + sub + lanes * i) * N, (c + sub + lanes * i) * WORD < row_bytes);
        for (uint32_t k = 0; k < top_k; ++k) {
            const int32_t r = row_of(k);
            if (r < 0) continue;
            uint16_t *dst = reinterpret_cast<uint16_t *>(rows + (size_t)r * stride);
#pragma unroll
            for (int i = 0; i < SEG_WORDS; ++i)
                if ((c + sub + lanes * i) * WORD < row_bytes) store_pack(dst + (c + sub + lanes * i) * N, v[i]);
        }
    } else {
        const uint32_t at = c * 16, bytes = on && at < row_bytes ? min(SEG_WORDS * lanes * 16, row_bytes - at) : 0;
        const uint32_t a = (uint32_t)reinterpret_cast<uintptr_t>(src + at) & 15;
        const uint32_t *q = reinterpret_cast<const uint32_t *>(src + at - a);
        Pack<uint32_t, 4> v[SEG_WORDS + 1];
#pragma unroll
        for (int i = 0; i <= SEG_WORDS; ++i) {  // the words that hold the part, one more than its units where it is not aligned
            const uint32_t w = sub + lanes * i;
            v[i] = load_pack_if<uint32_t, 4>(q + 4 * w, bytes && w * 16 < a + bytes && (i < SEG_WORDS || sub == 0));
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i <= SEG_WORDS; ++i)
            if (i < SEG_WORDS || sub == 0) *reinterpret_cast<Pack<uint32_t, 4> *>(st + 16 * (sub + lanes * i)) = v[i];
        __syncwarp();
        for (uint32_t k = 0; k < top_k; ++k) {
            const int32_t r = bytes ? row_of(k) : -1;
            if (r >= 0) write_part(rows + (size_t)r * stride + at, st, a, bytes, sub, lanes);
        }
    }
}

struct TileParams {
    const void *ids;
    int id_bytes;
    int64_t first;
    uint32_t experts, top_k, align;
    uint32_t inside;  // experts that an id can name: all, but for ids_from
    uint32_t num_slots, num_tokens, tile_tokens;
    uint32_t num_rows;
    int32_t *slot_of_row, *row_of_slot, *offsets, *counts;
    // counts of the tiles before, in two parts: of the group's tiles, [tiles][experts], and of the groups before
    const uint32_t *tile_before, *group_before;
    const uint32_t *totals;  // [experts]
    const unsigned char *x;       // nullptr: no rows
    unsigned char *rows;
    size_t x_stride, rows_stride;  // bytes
    uint32_t row_bytes, words;     // words: or units of 16 bytes, the last one perhaps not whole
    uint32_t log_lanes;            // 2^log_lanes lanes share a row: 32, or fewer for shorter rows
    uint32_t *error;               // the work buffer's error word
};

// Exclusive sums over the experts of the rounded and of the plain counts:
// offs[e] (rows before expert e) and pads[e] (rows without a slot before
// expert e), e = 0 .. experts.  One CTA; total[] may alias nothing.
template <int THREADS> __device__ __forceinline__ void expert_offsets(const uint32_t *total, uint32_t *offs, uint32_t *pads, uint32_t experts, uint32_t align) {
    __shared__ uint32_t warp_rows[THREADS / 32], warp_slots[THREADS / 32];
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t per = (experts + THREADS - 1) / THREADS;
    const uint32_t e0 = min(tid * per, experts), e1 = min(e0 + per, experts);
    uint32_t rows = 0, slots = 0;
    for (uint32_t e = e0; e < e1; ++e) {
        rows += (total[e] + align - 1) / align * align;
        slots += total[e];
    }
    uint32_t r = rows, s = slots;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t a = __shfl_up_sync(~0u, r, d), b = __shfl_up_sync(~0u, s, d);
        if (lane >= (uint32_t)d) {
            r += a;
            s += b;
        }
    }
    if (lane == 31) {
        warp_rows[warp] = r;
        warp_slots[warp] = s;
    }
    __syncthreads();
    r -= rows;
    s -= slots;
    for (uint32_t w = 0; w < warp; ++w) {
        r += warp_rows[w];
        s += warp_slots[w];
    }
    for (uint32_t e = e0; e < e1; ++e) {
        offs[e] = r;
        pads[e] = r - s;
        r += (total[e] + align - 1) / align * align;
        s += total[e];
    }
    if (tid == THREADS - 1) {  // the last thread's chunk ends at `experts`
        offs[experts] = r;
        pads[experts] = r - s;
    }
    __syncthreads();
}

// tile_counts[tile][e] becomes the count of bin e in the tiles before;
// totals[e] its count in all tiles.  A CTA takes 32 bins (a lane each), its
// warps share the tiles.
constexpr int SCAN_THREADS = 1024;
__global__ void __launch_bounds__(SCAN_THREADS) tile_scan_kernel(uint32_t *tile_counts, uint32_t *totals, uint32_t tiles,
                                                                   uint32_t bins) {
    __shared__ uint32_t sums[SCAN_THREADS / 32][32];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    const uint32_t a = (uint32_t)((uint64_t)tiles * warp / 32), b = (uint32_t)((uint64_t)tiles * (warp + 1) / 32);
    uint32_t sum = 0;
    wait_for_earlier();
    let_next_launch();
    if (e < bins) {
#pragma unroll 8
        for (uint32_t t = a; t < b; ++t) sum += tile_counts[(size_t)t * bins + e];
    }
    sums[warp][lane] = sum;
    __syncthreads();
    uint32_t before = 0;
    for (uint32_t w = 0; w < warp; ++w) before += sums[w][lane];
    if (e < bins) {
        if (warp == 31) totals[e] = before + sum;
#pragma unroll 8
        for (uint32_t t = a; t < b; ++t) {
            const uint32_t c = tile_counts[(size_t)t * bins + e];
            tile_counts[(size_t)t * bins + e] = before;
            before += c;
        }
    }
}

// One tile of tokens: the rows of its slots, then the tile's row movement.
// COUNT_HERE: the CTA counts every slot of the call itself; otherwise the
// counts of the tiles before it are in the work buffer.
//
// The movement is bound by DRAM, what comes before it by latency: reading the
// ids, shared atomics, the experts' sums and the ranks follow one another, 6.2 us
// for 8190 slots in a launch of their own.  4095 tokens of 8 KB, twice each, in
// tiles of 128 rows: 24 us, 4.4 TB/s, where the movement alone takes 21.
template <int WORD, bool COUNT_HERE, typename ID> __global__ void __launch_bounds__(COUNT_HERE ? HERE_THREADS : TILE_THREADS)
    expert_tile_kernel(const TileParams p) {
    constexpr int THREADS = COUNT_HERE ? HERE_THREADS : TILE_THREADS, WARPS = THREADS / 32;
    extern __shared__ __align__(16) unsigned char stage[];  // ODD_WORD: the warps' parts of rows; then the experts' arrays
    uint32_t *smem = reinterpret_cast<uint32_t *>(stage + (WORD == ODD_WORD ? WARPS * MOVE_STAGE : 0));
    const uint32_t E = p.experts;
    uint32_t *total = smem, *offs = total + E, *pads = offs + E + 1, *base = pads + E + 1;
    int32_t *row = reinterpret_cast<int32_t *>(base + E);
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t t0 = min(blockIdx.x * p.tile_tokens, p.num_tokens), t1 = min(t0 + p.tile_tokens, p.num_tokens);
    const uint32_t s0 = t0 * p.top_k, s1 = t1 * p.top_k;
    const ID *ids = static_cast<const ID *>(p.ids);
    const uint32_t lanes = 1u << p.log_lanes, seg_words = (uint32_t)SEG_WORDS << p.log_lanes, segs = (p.words + seg_words - 1) / seg_words;
    const uint32_t g0 = segs * blockIdx.y / gridDim.y, g1 = segs * (blockIdx.y + 1) / gridDim.y;  // the CTA's columns

    wait_for_earlier();
    for (uint32_t s = s0 + tid; s < s1; s += THREADS) row[s - s0] = id_index(ids, s, p.first, p.inside);  // the slots' experts, then their rows
    if (COUNT_HERE) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *p.error = 0;  // no wait here can run out
        for (uint32_t e = tid; e < E; e += THREADS) total[e] = base[e] = 0;
        __syncthreads();
#pragma unroll 8
        for (uint32_t s = tid; s < p.num_slots; s += THREADS) {
            const int32_t e = id_index(ids, s, p.first, p.inside);
            if (e >= 0) atomicAdd(s < s0 ? &base[e] : &total[e], 1u);
        }
        __syncthreads();
        for (uint32_t e = tid; e < E; e += THREADS) total[e] += base[e];
    } else {
        for (uint32_t e = tid; e < E; e += THREADS) {
            total[e] = p.totals[e];
            base[e] = p.tile_before[(size_t)blockIdx.x * E + e] + p.group_before[(size_t)(blockIdx.x / GROUP_TILES) * E + e];
        }
    }
    __syncthreads();
    expert_offsets<THREADS>(total, offs, pads, E, p.align);
    for (uint32_t e = tid; e < E; e += THREADS) base[e] += offs[e];
    __syncthreads();

    // stable ranks: one warp takes the tile's slots in order, 32 at a time
    if (warp == 0) {
        for (uint32_t s = s0; s < s1; s += 32) {
            const int32_t e = s + lane < s1 ? row[s + lane - s0] : -1;
            const uint32_t peers = __match_any_sync(~0u, e), below = __popc(peers & lanemask_lt());
            int32_t r = -1;
            if (e >= 0) r = (int32_t)(base[e] + below);
            __syncwarp();
            if (e >= 0 && below == 0) base[e] += __popc(peers);
            __syncwarp();
            if (s + lane < s1) {
                row[s + lane - s0] = r;
                if (blockIdx.y == 0) {
                    p.row_of_slot[s + lane] = r;
                    if (r >= 0) p.slot_of_row[r] = (int32_t)(s + lane);
                }
            }
        }
    } else if (blockIdx.y == 0 && blockIdx.x == 0) {
        for (uint32_t e = tid - 32; e <= E; e += THREADS - 32) {
            p.offsets[e] = (int32_t)offs[e];
            if (e < E) p.counts[e] = (int32_t)total[e];
        }
    }
    __syncthreads();

    if (p.x != nullptr && g1 > g0 && t1 > t0) {
        const uint32_t per_warp = 32 >> p.log_lanes, sub = lane & (lanes - 1);  // tokens of a warp's turn, lane of the row
        const uint32_t turns = (t1 - t0 + per_warp - 1) / per_warp * (g1 - g0);
        for (uint32_t u = warp; u < turns; u += WARPS) {
            const uint32_t which = lane >> p.log_lanes, t = u / (g1 - g0) * per_warp + which, c = (g0 + u % (g1 - g0)) * seg_words;
            const bool on = t < t1 - t0;
            move_segment<WORD>(p.x + (t0 + (on ? t : 0)) * p.x_stride, c, sub, lanes, p.row_bytes, on, p.top_k,
                              [&](uint32_t k) { return row[t * p.top_k + k]; }, p.rows, p.rows_stride,
                              WORD == ODD_WORD ? stage + warp * MOVE_STAGE + which * (seg_words * 16 + PART_PAD) : nullptr);
        }
    }
    // rows without a slot: the j-th of them follows expert e's rows, with e
    // the last expert that has at most j such rows before it; neighbours go to
    // different CTAs
    const uint32_t holes = p.num_rows - (offs[E] - pads[E]);
    for (uint32_t j = warp * gridDim.x + blockIdx.x; j < holes; j += gridDim.x * WARPS) {
        uint32_t lo = 0, hi = E;
        while (lo < hi) {
            const uint32_t mid = (lo + hi + 1) / 2;
            if (pads[mid] <= j) lo = mid;
            else hi = mid - 1;
        }
        const uint32_t r = offs[lo] + (lo < E ? total[lo] : 0u) + (j - pads[lo]);
        if (blockIdx.y == 0 && lane == 0) p.slot_of_row[r] = -1;
        if (p.x != nullptr && g1 > g0) {
            const uint32_t unit = unit_bytes(WORD), at = g0 * seg_words * unit;
            zero_bytes(p.rows + (size_t)r * p.rows_stride + at, min(g1 * seg_words * unit, p.row_bytes) - at);
        }
    }
}

// Counts of every expert: each of the CTA's warps takes a tile.  tile_before
// gets the counts of the group's tiles before each, group_counts the group's.
template <typename ID> __global__ void __launch_bounds__(32 * GROUP_TILES) expert_count_kernel(const TileParams p, uint32_t tiles, uint32_t *tile_before,
                                                                                          uint32_t *group_counts) {
    extern __shared__ uint32_t smem[];  // [GROUP_TILES][experts]
    const uint32_t E = p.experts, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tile = blockIdx.x * GROUP_TILES + warp;
    for (uint32_t e = threadIdx.x; e < GROUP_TILES * E; e += 32 * GROUP_TILES) smem[e] = 0;
    wait_for_earlier();
    let_next_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.error = 0;
    __syncthreads();
    const uint64_t slots = (uint64_t)p.tile_tokens * p.top_k, a = tile * slots, b = min(a + slots, (uint64_t)p.num_slots);
#pragma unroll 8
    for (uint64_t s = a + lane; s < b; s += 32) {
        const int32_t e = id_index(static_cast<const ID *>(p.ids), s, p.first, p.inside);
        if (e >= 0) atomicAdd(&smem[warp * E + e], 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < E; e += 32 * GROUP_TILES) {
        uint32_t sum = 0;
#pragma unroll
        for (uint32_t w = 0; w < GROUP_TILES; ++w) {
            if (blockIdx.x * GROUP_TILES + w < tiles) tile_before[(size_t)(blockIdx.x * GROUP_TILES + w) * E + e] = sum;
            sum += smem[w * E + e];
        }
        group_counts[(size_t)blockIdx.x * E + e] = sum;
    }
}

uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Tokens of a tile whose counts are in the work buffer.
uint32_t tile_tokens_of(size_t num_slots, size_t top_k) {
    size_t slots = num_slots > LONG_SLOTS ? TILE_SLOTS_LONG : TILE_SLOTS;
    while (slots > TILE_SLOTS_LEAST && num_slots / slots < 152 * 8) slots /= 2;
    return (uint32_t)(top_k >= slots ? 1 : slots / top_k);
}

// log2 of the lanes that share a row of `words` words.
uint32_t log_lanes_of(uint32_t words, bool any) {
    uint32_t log_lanes = any ? ODD_LOG_LANES : 0;
    while ((1u << log_lanes) < words && log_lanes < 5) ++log_lanes;
    return log_lanes;
}

template <int WORD, typename ID> cudaError_t launch_tiles_of(const ExpertJob &job, TileParams p, cudaStream_t stream, int *launches) {
    const bool count_here = p.num_slots <= COUNT_HERE_SLOTS;
    const uint32_t sms = (uint32_t)device_sm_count();
    p.tile_tokens = count_here ? max_u32((p.num_tokens + 2 * sms - 1) / (2 * sms), 1) : tile_tokens_of(p.num_slots, p.top_k);
    uint32_t tiles = (p.num_tokens + p.tile_tokens - 1) / p.tile_tokens;
    cudaError_t e = cudaSuccess;
    if (!count_here) {
        const uint32_t groups = (tiles + GROUP_TILES - 1) / GROUP_TILES;
        uint32_t *group_counts = job.tile_counts + (size_t)tiles * p.experts, *totals = group_counts + (size_t)groups * p.experts;
        e = launch_next(expert_count_kernel<ID>, groups, 32 * GROUP_TILES, GROUP_TILES * p.experts * sizeof(uint32_t), stream, p, tiles,
                        job.tile_counts, group_counts);
        if (e != cudaSuccess) return e;
        ++*launches;
        timing_mark(stream);
        if ((e = launch_tile_scan(group_counts, totals, groups, p.experts, stream, launches)) != cudaSuccess) return e;
        p.tile_before = job.tile_counts;
        p.group_before = group_counts;
        p.totals = totals;
    }
    if (tiles == 0) tiles = 1;  // no tokens: the offsets and the empty rows are still written
    size_t smem = (4 * (size_t)p.experts + 2 + (size_t)p.tile_tokens * p.top_k) * sizeof(uint32_t);
    // few tiles: their rows are cut into columns, so that every SM moves some
    p.log_lanes = log_lanes_of(p.words, WORD == ODD_WORD);
    const uint32_t seg = (uint32_t)SEG_WORDS << p.log_lanes, segs = (p.words + seg - 1) / seg;
    uint32_t cols = 1;
    if (p.x != nullptr && tiles < sms) {
        cols = (segs * p.tile_tokens + 7) / 8;
        if (cols > 2 * sms / tiles) cols = 2 * sms / tiles;
        if (cols < 1) cols = 1;
    }
    // few tokens and many rows without a slot: more CTAs, without tokens, that zero them
    uint32_t all_tiles = tiles;
    if (count_here && p.num_rows - p.num_slots > 16 * tiles) {
        const uint32_t zeroing = (p.num_rows - p.num_slots + 15) / 16;
        all_tiles = max_u32(tiles, zeroing < 2 * sms ? zeroing : 2 * sms);
    }
    const dim3 grid(all_tiles, cols);
    if constexpr (WORD == ODD_WORD) {
        static PerDeviceOnce once;
        e = once.run([] {
            const int most = (int)(HERE_THREADS / 32 * MOVE_STAGE + 40 * 1024);
            const cudaError_t r = cudaFuncSetAttribute(expert_tile_kernel<WORD, true, ID>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
            return r != cudaSuccess ? r : cudaFuncSetAttribute(expert_tile_kernel<WORD, false, ID>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        });
        if (e != cudaSuccess) return e;
        smem += (size_t)(count_here ? HERE_THREADS : TILE_THREADS) / 32 * MOVE_STAGE;
    }
    if (count_here) e = launch_next(expert_tile_kernel<WORD, true, ID>, grid, HERE_THREADS, smem, stream, p);
    else e = launch_next(expert_tile_kernel<WORD, false, ID>, grid, TILE_THREADS, smem, stream, p);
    ++*launches;
    timing_mark(stream);
    return e;
}
template <int WORD> cudaError_t launch_tiles(const ExpertJob &job, const TileParams &p, cudaStream_t stream, int *launches) {
    return p.id_bytes == 8 ? launch_tiles_of<WORD, int64_t>(job, p, stream, launches)
                           : launch_tiles_of<WORD, int32_t>(job, p, stream, launches);
}

// Width of the words that rows move in: 16, 8, 4 or 2 bytes, or ODD_WORD.
int word_of(const Rows *rows, int count, size_t row_len) {
    const size_t bytes = (size_t)pack_values(rows, count, row_len) * row_bytes(rows[0].type);
    if (bytes == 2 && row_len * row_bytes(rows[0].type) >= ODD_BYTES) return ODD_WORD;
    return bytes > 16 ? 16 : (int)bytes;
}

// ---------------------------------------------------------------------------
// Gather by an existing plan
// ---------------------------------------------------------------------------

struct MoveParams {
    const int32_t *slot_of_row, *row_of_slot;
    const void *weights;
    void *d_weights;
    const unsigned char *x;
    unsigned char *out, *rows, *d_rows;
    size_t x_stride, rows_stride, d_rows_stride;  // bytes
    uint32_t num_tokens, top_k, num_rows;
    uint32_t zero_rows, zero_units;  // rows that a warp looks at for empty ones; warps that do
    uint32_t row_len, row_bytes, packs, segs, steps, log_lanes;  // packs of 16 bytes, the last one perhaps not whole
};

constexpr int MOVE_THREADS = 256;
constexpr int MOVE_WARPS = MOVE_THREADS / 32;

// Zeroes those of up to p.zero_rows rows, p.zero_units apart from `unit` on, that
// hold no slot; a warp's work.  Such rows are neighbours: a stride gives every CTA
// some (4095 tokens to 9216 rows of 8 KB 21 us; side by side 24).
__device__ __forceinline__ void zero_rows_without_slot(const MoveParams &p, uint64_t unit, unsigned char *rows, size_t stride) {
    const uint32_t lane = threadIdx.x & 31;
    const uint64_t mine = unit + (uint64_t)lane * p.zero_units;
    uint32_t holes = __ballot_sync(~0u, lane < p.zero_rows && mine < p.num_rows && p.slot_of_row[mine] < 0);
    while (holes) {
        const uint64_t r = unit + (uint64_t)(__ffs(holes) - 1) * p.zero_units;
        holes &= holes - 1;
        zero_bytes(rows + r * stride, p.row_bytes);
    }
}

// A warp takes a segment of one token's row (of several tokens' where rows
// are short), or p.zero_rows rows to look for empty ones.  Each byte is read
// once and written top_k times; 65536 tokens of 4 KB to 8 rows each 361 us, the
// 2.4 GB at 6.7 TB/s.
template <int WORD> __global__ void __launch_bounds__(MOVE_THREADS) expert_gather_kernel(const MoveParams p) {
    const uint32_t lane = threadIdx.x & 31, lanes = 1u << p.log_lanes, per_warp = 32 >> p.log_lanes;
    const uint64_t u = (uint64_t)blockIdx.x * MOVE_WARPS + (threadIdx.x >> 5);
    const uint64_t units = (uint64_t)((p.num_tokens + per_warp - 1) / per_warp) * p.segs;
    wait_for_earlier();
    if (u >= units) {
        if (u - units < p.zero_units) zero_rows_without_slot(p, u - units, p.rows, p.rows_stride);
        return;
    }
    const uint32_t which = lane >> p.log_lanes, t = (uint32_t)(u / p.segs) * per_warp + which, c = (uint32_t)(u % p.segs) * lanes * SEG_WORDS;
    const bool on = t < p.num_tokens;
    __shared__ __align__(16) unsigned char stage[WORD == ODD_WORD ? MOVE_WARPS * MOVE_STAGE : 16];
    move_segment<WORD>(p.x + (on ? t : 0) * p.x_stride, c, lane & (lanes - 1), lanes, p.row_bytes, on, p.top_k, [&](uint32_t k) {
        const int32_t r = p.row_of_slot[(size_t)t * p.top_k + k];
        return (uint32_t)r < p.num_rows ? r : -1;
    }, p.rows, p.rows_stride, WORD == ODD_WORD ? stage + (threadIdx.x >> 5) * MOVE_STAGE + which * (SEG_WORDS * lanes * 16 + PART_PAD) : nullptr);
}

// ---------------------------------------------------------------------------
// Combine
// ---------------------------------------------------------------------------

// A warp takes a token's segment of p.steps * 32 packs at a time.  Lane
// k holds slot k's row and weight (top_k above 32: in turns of 32), fetched
// one segment ahead of the rows, so that the rows' loads wait for no index.
// The slots are summed in the order of k in 32 bits, U rows in flight: 24
// warps an SM with 4 KB each cover DRAM's latency.  Bound by the rows' bytes:
// 16384 tokens of 8 KB, 6 slots of 8 with a row, 144 us, 6.5 TB/s.
constexpr uint32_t COMBINE_STEPS = 4, COMBINE_STEPS_ODD = 8;  // at most
template <typename T, typename W, bool ODD, int U> __global__ void __launch_bounds__(MOVE_THREADS, 3) expert_combine_kernel(const MoveParams p) {
    constexpr int N = 16 / (int)sizeof(T);
    const uint32_t lane = threadIdx.x & 31;
    __shared__ __align__(16) unsigned char stage[ODD ? MOVE_WARPS : 1][ODD ? COMBINE_STEPS_ODD * 512 + PART_PAD : 16];
    unsigned char *st = stage[ODD ? threadIdx.x >> 5 : 0];
    const uint64_t units = (uint64_t)p.num_tokens * p.segs, stride = (uint64_t)gridDim.x * MOVE_WARPS;
    const W *weights = static_cast<const W *>(p.weights);
    const uint32_t first = min(p.top_k, 32u);
    wait_for_earlier();
    uint64_t u = (uint64_t)blockIdx.x * MOVE_WARPS + (threadIdx.x >> 5);
    int32_t row = -1;
    float weight = 0.0f;
    if (u < units && lane < first) {
        row = p.row_of_slot[u / p.segs * p.top_k + lane];
        weight = weight_at(weights, u / p.segs * p.top_k + lane);
    }
    for (; u < units; u += stride) {
        const uint64_t t = u / p.segs, next = (u + stride) / p.segs;
        const uint32_t c0 = ((uint32_t)(u % p.segs) * p.steps * 32 + lane) * N;
        const int32_t row_now = (uint32_t)row < p.num_rows ? row : -1;
        const float weight_now = weight;
        if (u + stride < units && lane < first) {
            row = p.row_of_slot[next * p.top_k + lane];
            weight = weight_at(weights, next * p.top_k + lane);
        }
#pragma unroll 1
        for (uint32_t step = 0; step < p.steps; ++step) {
            const uint32_t c = c0 + step * 32 * N;
            if (c - lane * N >= p.row_len) break;  // the same for the whole warp
            float acc[N] = {};
            for (uint32_t k0 = 0; k0 < p.top_k; k0 += U) {
                int32_t r32 = row_now;
                float w32 = weight_now;
                if (k0 >= 32) {
                    const uint32_t k = (k0 & ~31u) + lane;
                    r32 = k < p.top_k ? p.row_of_slot[t * p.top_k + k] : -1;
                    if ((uint32_t)r32 >= p.num_rows) r32 = -1;
                    w32 = k < p.top_k ? weight_at(weights, t * p.top_k + k) : 0.0f;
                }
                Pack<T, N> v[U];
                float w[U];
                int32_t r[U];
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    r[j] = __shfl_sync(~0u, r32, (k0 + j) & 31);
                    w[j] = __shfl_sync(~0u, w32, (k0 + j) & 31);
                }
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const bool on = r[j] >= 0 && k0 + j < p.top_k;
                    if (!on) w[j] = 0.0f;
                    v[j] = load_row<ODD>(reinterpret_cast<const T *>(p.rows + (int64_t)r[j] * (int64_t)p.rows_stride), c, p.row_len, on);
                }
#pragma unroll
                for (int j = 0; j < U; ++j)
#pragma unroll
                    for (int i = 0; i < N; ++i) acc[i] = fmaf(w[j], to_f32(v[j].v[i]), acc[i]);
            }
            Pack<T, N> o;
#pragma unroll
            for (int i = 0; i < N; ++i) o.v[i] = from_f32<T>(acc[i]);
            put_pack<ODD>(reinterpret_cast<T *>(p.out + t * p.x_stride), c, p.row_len, o, true, st, step * 32 + lane);
        }
        if (ODD) {
            const uint32_t c1 = c0 - lane * N;
            __syncwarp();
            write_part(p.out + t * p.x_stride + c1 * sizeof(T), st, 0, part_bytes<T>(c1, p.steps * 32 * N, p.row_len), lane, 32);
            __syncwarp();
        }
    }
}

// The same for rows of fewer than 32 packs: 2^p.log_lanes lanes take a token, each
// with its own loads of the token's indices.
template <typename T, typename W, bool ODD, int U> __global__ void __launch_bounds__(MOVE_THREADS, 3) expert_combine_short_kernel(const MoveParams p) {
    const uint64_t t = ((uint64_t)blockIdx.x * MOVE_THREADS + threadIdx.x) >> p.log_lanes;
    constexpr int N = 16 / (int)sizeof(T);
    const uint32_t lanes = 1u << p.log_lanes, c = (threadIdx.x & (lanes - 1)) * N;
    const bool here = t < p.num_tokens;
    wait_for_earlier();
    if (!ODD && (!here || c >= p.row_len)) return;
    const W *weights = static_cast<const W *>(p.weights);
    float acc[N] = {};
    for (uint32_t k0 = 0; k0 < p.top_k; k0 += U) {
        Pack<T, N> v[U];
        float w[U];
        int32_t r[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            r[j] = here && k0 + j < p.top_k ? p.row_of_slot[t * p.top_k + k0 + j] : -1;
            w[j] = here && k0 + j < p.top_k ? weight_at(weights, t * p.top_k + k0 + j) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const bool on = (uint32_t)r[j] < p.num_rows;
            if (!on) w[j] = 0.0f;
            v[j] = load_row<ODD>(reinterpret_cast<const T *>(p.rows + (int64_t)r[j] * (int64_t)p.rows_stride), c, p.row_len, on);
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(w[j], to_f32(v[j].v[i]), acc[i]);
    }
    Pack<T, N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.v[i] = from_f32<T>(acc[i]);
    constexpr uint32_t STAGE = 32 * 16 + (32 >> ODD_LOG_LANES) * PART_PAD;
    __shared__ __align__(16) unsigned char stage[ODD ? MOVE_WARPS * STAGE : 16];
    const uint32_t which = (threadIdx.x & 31) >> p.log_lanes;
    unsigned char *st = stage + (ODD ? (threadIdx.x >> 5) * STAGE + which * (lanes * 16 + PART_PAD) : 0);
    put_pack<ODD>(reinterpret_cast<T *>(p.out + (here ? t : 0) * p.x_stride), c, p.row_len, o, here, st, threadIdx.x & (lanes - 1));
    if (ODD) {
        __syncwarp();
        if (here) write_part(p.out + t * p.x_stride, st, 0, p.row_bytes, threadIdx.x & (lanes - 1), lanes);
    }
}

// ---------------------------------------------------------------------------
// Combine's gradient
// ---------------------------------------------------------------------------

// A warp takes one slot: its row of d_rows and its weight's gradient, a dot
// product summed in 32 bits by lane and then over the lanes in a fixed order.
// The slots of a token follow one another, so that d_out's row is read from
// DRAM once.  Bound by the rows' bytes, one read and one write for three
// operations a value: 16384 tokens of 8 slots of 8 KB 330 us, 6.9 TB/s, with four
// CTAs an SM and predicated loads; three CTAs with branches 353.
template <typename T, typename W, int N> __global__ void __launch_bounds__(MOVE_THREADS, 4) expert_combine_grad_kernel(const MoveParams p) {
    const uint32_t lane = threadIdx.x & 31;
    const uint64_t u = (uint64_t)blockIdx.x * MOVE_WARPS + (threadIdx.x >> 5);
    const uint64_t slots = (uint64_t)p.num_tokens * p.top_k;
    wait_for_earlier();
    if (u >= slots) {
        if (u - slots < p.zero_units) zero_rows_without_slot(p, u - slots, p.d_rows, p.d_rows_stride);
        return;
    }
    W *d_weights = static_cast<W *>(p.d_weights);
    const int32_t r = p.row_of_slot[u];
    if ((uint32_t)r >= p.num_rows) {
        if (d_weights && lane == 0) d_weights[u] = from_f32<W>(0.0f);
        return;
    }
    const float w = weight_at(static_cast<const W *>(p.weights), u);
    const T *d_out = reinterpret_cast<const T *>(p.x + (u / p.top_k) * p.x_stride);
    const T *y = reinterpret_cast<const T *>(p.rows + (size_t)r * p.rows_stride);
    T *d_row = reinterpret_cast<T *>(p.d_rows + (size_t)r * p.d_rows_stride);
    float dot = 0.0f;
    constexpr int U = 4;
    for (uint32_t c0 = lane * N; c0 < p.row_len; c0 += 32 * N * U) {
        Pack<T, N> d[U], v[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t c = c0 + 32 * N * j;
            d[j] = load_pack_if<T, N>(d_out + c, c < p.row_len);
            v[j] = load_pack_if<T, N>(y + c, d_weights && c < p.row_len);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t c = c0 + 32 * N * j;
            Pack<T, N> o;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float g = to_f32(d[j].v[i]);
                o.v[i] = from_f32<T>(w * g);
                dot = fmaf(g, to_f32(v[j].v[i]), dot);
            }
            if (c < p.row_len) store_pack(d_row + c, o);
        }
    }
#pragma unroll
    for (int s = 16; s > 0; s /= 2) dot += __shfl_xor_sync(~0u, dot, s);
    if (d_weights && lane == 0) d_weights[u] = from_f32<W>(dot);
}

// The same for rows of at most GRAD_SHORT packs, where a slot has too few
// bytes to hide its indices: a warp's turn is GRAD_PACKS / p.steps slots for
// every 2^p.log_lanes lanes, with the next turn's indices fetched ahead (lane l holds
// the turn's l-th slot).  240000 slots of 31 packs: 83 us, a warp per slot 180;
// of 65 packs: 232 against 194.
constexpr int GRAD_PACKS = 4;
constexpr uint32_t GRAD_SHORT = 64;
template <typename T, typename W, int N> __global__ void __launch_bounds__(MOVE_THREADS, 3) expert_combine_grad_short_kernel(const MoveParams p) {
    constexpr int U = GRAD_PACKS;
    const uint32_t lane = threadIdx.x & 31, lanes = 1u << p.log_lanes, sub = lane & (lanes - 1), which = lane >> p.log_lanes, per_warp = 32 >> p.log_lanes;
    const uint32_t log_steps = __ffs(p.steps) - 1, turn = (U >> log_steps) * per_warp;  // slots of a turn, at most 32
    const uint64_t slots = (uint64_t)p.num_tokens * p.top_k, turns = (slots + turn - 1) / turn;
    const uint64_t warp = (uint64_t)blockIdx.x * MOVE_WARPS + (threadIdx.x >> 5), warps = (uint64_t)gridDim.x * MOVE_WARPS;
    const W *weights = static_cast<const W *>(p.weights);
    W *d_weights = static_cast<W *>(p.d_weights);
    wait_for_earlier();
    int32_t next_row = -1;
    float next_weight = 0.0f;
    if (lane < turn && warp * turn + lane < slots) {
        next_row = p.row_of_slot[warp * turn + lane];
        next_weight = weight_at(weights, warp * turn + lane);
    }
    for (uint64_t t = warp; t < turns; t += warps) {
        const int32_t row = (uint32_t)next_row < p.num_rows ? next_row : -1;
        const float weight = next_weight;
        const uint64_t ahead = (t + warps) * turn + lane;
        next_row = -1;
        if (lane < turn && ahead < slots) {
            next_row = p.row_of_slot[ahead];
            next_weight = weight_at(weights, ahead);
        }
        Pack<T, N> d[U], v[U];
        int32_t r[U];
        float w[U], dot[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            r[j] = __shfl_sync(~0u, row, (j >> log_steps) * per_warp + which);
            w[j] = __shfl_sync(~0u, weight, (j >> log_steps) * per_warp + which);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint64_t slot = t * turn + (j >> log_steps) * per_warp + which;
            const uint32_t c = ((j & (p.steps - 1)) * lanes + sub) * N;
            const bool on = r[j] >= 0 && c < p.row_len;
            d[j] = load_pack_if<T, N>(reinterpret_cast<const T *>(p.x + (on ? slot / p.top_k : 0) * p.x_stride) + c, on);
            v[j] = load_pack_if<T, N>(reinterpret_cast<const T *>(p.rows + (on ? (size_t)r[j] : 0) * p.rows_stride) + c, on && d_weights);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t c = ((j & (p.steps - 1)) * lanes + sub) * N;
            Pack<T, N> o;
            dot[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float g = to_f32(d[j].v[i]);
                o.v[i] = from_f32<T>(w[j] * g);
                dot[j] = fmaf(g, to_f32(v[j].v[i]), dot[j]);
            }
            if (r[j] >= 0 && c < p.row_len) store_pack(reinterpret_cast<T *>(p.d_rows + (size_t)r[j] * p.d_rows_stride) + c, o);
        }
        if (d_weights == nullptr) continue;
        if (p.steps == 2) dot[0] += dot[1], dot[2] += dot[3];  // a slot's packs lie in neighbouring j
#pragma unroll
        for (int j = 0; j < U; ++j) {
            for (uint32_t s = lanes / 2; s > 0; s /= 2) dot[j] += __shfl_xor_sync(~0u, dot[j], s);
            const uint64_t slot = t * turn + (j >> log_steps) * per_warp + which;
            if ((j & (p.steps - 1)) == 0 && sub == 0 && slot < slots) d_weights[slot] = from_f32<W>(dot[j]);
        }
    }
    for (uint64_t unit = warp; unit < p.zero_units; unit += warps) zero_rows_without_slot(p, unit, p.d_rows, p.d_rows_stride);
}

MoveParams move_params(const ExpertMoveJob &job) {
    MoveParams p = {};
    const size_t b = (size_t)row_bytes(job.rows.type);
    p.slot_of_row = job.slot_of_row;
    p.row_of_slot = job.row_of_slot;
    p.weights = job.weights;
    p.d_weights = job.d_weights;
    p.x = static_cast<const unsigned char *>(job.x.base);
    p.out = static_cast<unsigned char *>(job.x.base);
    p.rows = static_cast<unsigned char *>(job.rows.base);
    p.d_rows = static_cast<unsigned char *>(job.d_rows.base);
    p.x_stride = job.x.stride * b;
    p.rows_stride = job.rows.stride * b;
    p.d_rows_stride = job.d_rows.stride * b;
    p.num_tokens = (uint32_t)job.num_tokens;
    p.top_k = job.top_k;
    p.num_rows = (uint32_t)job.num_rows;
    p.row_len = (uint32_t)job.row_len;
    p.row_bytes = (uint32_t)(job.row_len * b);
    // few long ones to a warp: rows of 8 KB, 11% of them empty, 21 us with 4, 23 with 8; of 2 KB, 6%, 51 and 49; of 200
    // bytes, 6%, 12.3 with 4 and 11.0 with 32
    p.zero_rows = p.row_bytes >= 8192 ? 4 : p.row_bytes >= 1024 ? 8 : 32;
    p.zero_units = (p.num_rows + p.zero_rows - 1) / p.zero_rows;
    p.packs = (p.row_bytes + 15) / 16;
    return p;
}

template <typename T, typename W, bool ODD> cudaError_t launch_combine(const MoveParams &p0, cudaStream_t stream) {
    MoveParams p = p0;
    if (p.packs < 32) {
        p.log_lanes = log_lanes_of(p.packs, ODD);
        const unsigned grid = (unsigned)((((uint64_t)p.num_tokens << p.log_lanes) + MOVE_THREADS - 1) / MOVE_THREADS);
        return launch_next(p.top_k <= 2 ? expert_combine_short_kernel<T, W, ODD, 2> : expert_combine_short_kernel<T, W, ODD, 8>, grid, MOVE_THREADS, 0,
                           stream, p);
    }
    // longer segments reuse a token's indices (and have fewer ends); short ones give every warp work when there are few tokens
    const uint32_t most_warps = (uint32_t)device_sm_count() * 3 * MOVE_WARPS;
    p.steps = ODD ? COMBINE_STEPS_ODD : COMBINE_STEPS;
    while (p.steps > 1 && (uint64_t)p.num_tokens * ((p.packs + 32 * p.steps - 1) / (32 * p.steps)) < 2 * most_warps) p.steps /= 2;
    p.segs = (p.packs + 32 * p.steps - 1) / (32 * p.steps);
    p.steps = (p.packs + 32 * p.segs - 1) / (32 * p.segs);  // segments of equal length
    const uint64_t blocks = ((uint64_t)p.num_tokens * p.segs + MOVE_WARPS - 1) / MOVE_WARPS;
    const unsigned most = (unsigned)device_sm_count() * 3, grid = blocks < most ? (unsigned)blocks : most;
    const auto kernel = p.top_k <= 2   ? expert_combine_kernel<T, W, ODD, 2>
                        : p.top_k <= 4 ? expert_combine_kernel<T, W, ODD, 4>
                                       : expert_combine_kernel<T, W, ODD, 8>;
    return launch_next(kernel, grid, MOVE_THREADS, 0, stream, p);
}

template <typename T, typename W, int N> cudaError_t launch_combine_grad(const MoveParams &p0, cudaStream_t stream) {
    MoveParams p = p0;
    p.packs = p.row_len / N;
    const uint64_t holes = p.zero_units;
    if (p.packs <= GRAD_SHORT) {
        p.log_lanes = log_lanes_of(p.packs, false);
        p.steps = p.packs > 32 ? 2 : 1;
        while (GRAD_PACKS / p.steps * (32 >> p.log_lanes) > 32) ++p.log_lanes;  // a lane holds each slot of a turn
        const uint32_t turn = GRAD_PACKS / p.steps * (32 >> p.log_lanes);
        const uint64_t turns = ((uint64_t)p.num_tokens * p.top_k + turn - 1) / turn;
        const uint64_t blocks = ((turns > holes ? turns : holes) + MOVE_WARPS - 1) / MOVE_WARPS, most = (uint64_t)device_sm_count() * 3;
        return launch_next(expert_combine_grad_short_kernel<T, W, N>, (unsigned)(blocks < most ? blocks : most), MOVE_THREADS, 0, stream, p);
    }
    const uint64_t units = (uint64_t)p.num_tokens * p.top_k + holes;
    return launch_next(expert_combine_grad_kernel<T, W, N>, (unsigned)((units + MOVE_WARPS - 1) / MOVE_WARPS), MOVE_THREADS, 0, stream, p);
}

// The gradient has few operations to spare for cutting packs out of words, and
// takes the widest packs that its rows allow: 16 bytes, two values or one.
// (240000 slots of 1082 bf16 values: 199 us by twos; through aligned words 410.)
template <typename T, typename W> cudaError_t launch_move(const MoveParams &p, bool grad, int n, cudaStream_t stream) {
    constexpr int FULL = 16 / (int)sizeof(T);
    if (!grad) return n >= FULL ? launch_combine<T, W, false>(p, stream) : launch_combine<T, W, true>(p, stream);
    if (n >= FULL) return launch_combine_grad<T, W, FULL>(p, stream);
    return n >= 2 ? launch_combine_grad<T, W, 2>(p, stream) : launch_combine_grad<T, W, 1>(p, stream);
}

cudaError_t launch_gather(const ExpertMoveJob &job, cudaStream_t stream, int *launches) {
    MoveParams p = move_params(job);
    const Rows rows[2] = {job.x, job.rows};
    const int word = word_of(rows, 2, job.row_len);
    p.packs = (p.row_bytes + unit_bytes(word) - 1) / unit_bytes(word);
    p.log_lanes = log_lanes_of(p.packs, word == ODD_WORD);
    const uint32_t seg = (uint32_t)SEG_WORDS << p.log_lanes, per_warp = 32 >> p.log_lanes;
    p.segs = (p.packs + seg - 1) / seg;
    const uint64_t units = (uint64_t)((p.num_tokens + per_warp - 1) / per_warp) * p.segs + p.zero_units;
    if (units > (uint64_t)MOVE_WARPS * 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    const unsigned blocks = (unsigned)((units + MOVE_WARPS - 1) / MOVE_WARPS);
    const auto kernel = word == 16  ? expert_gather_kernel<16>
                        : word == 8 ? expert_gather_kernel<8>
                        : word == 4 ? expert_gather_kernel<4>
                        : word == 2 ? expert_gather_kernel<2>
                                    : expert_gather_kernel<ODD_WORD>;
    const cudaError_t e = launch_next(kernel, blocks, MOVE_THREADS, 0, stream, p);
    ++*launches;
    timing_mark(stream);
    return e;
}

cudaError_t launch_typed(const ExpertMoveJob &job, bool grad, cudaStream_t stream, int *launches) {
    const Rows rows[3] = {job.x, job.rows, job.d_rows};
    const int n = pack_values(rows, grad ? 3 : 2, job.row_len);
    const MoveParams p = move_params(job);
    cudaError_t e;
    const bool w32 = job.weight_type == ROW_F32;
    if (job.rows.type == ROW_F32) e = launch_move<float, float>(p, grad, n, stream);
    else if (job.rows.type == ROW_F16) e = w32 ? launch_move<__half, float>(p, grad, n, stream)
                                               : launch_move<__half, __half>(p, grad, n, stream);
    else e = w32 ? launch_move<__nv_bfloat16, float>(p, grad, n, stream)
                 : launch_move<__nv_bfloat16, __nv_bfloat16>(p, grad, n, stream);
    ++*launches;
    timing_mark(stream);
    return e;
}

}  // namespace

cudaError_t launch_tile_scan(uint32_t *tile_counts, uint32_t *totals, uint32_t tiles, uint32_t bins, cudaStream_t stream,
                             int *launches) {
    const cudaError_t e = launch_next(tile_scan_kernel, (bins + 31) / 32, SCAN_THREADS, 0, stream, tile_counts, totals, tiles, bins);
    ++*launches;
    timing_mark(stream);
    return e;
}

size_t expert_temp_bytes(size_t num_tokens, size_t top_k, size_t num_experts) {
    const size_t slots = num_tokens * top_k;
    if (slots <= COUNT_HERE_SLOTS) return 0;
    const size_t per = tile_tokens_of(slots, top_k), tiles = (num_tokens + per - 1) / per;
    return (tiles + (tiles + GROUP_TILES - 1) / GROUP_TILES + 1) * num_experts * sizeof(uint32_t);
}

cudaError_t launch_expert_dispatch(const ExpertJob &job, cudaStream_t stream, int *launches) {
    TileParams p = {};
    p.ids = job.ids;
    p.id_bytes = job.id_bytes;
    p.first = job.first_expert;
    p.experts = job.num_experts;
    p.inside = (uint32_t)ids_from(job.first_expert, job.num_experts);
    p.top_k = job.top_k;
    p.align = job.row_align;
    p.num_tokens = (uint32_t)job.num_tokens;
    p.num_slots = (uint32_t)(job.num_tokens * job.top_k);
    p.num_rows = (uint32_t)job.num_rows;
    p.slot_of_row = job.slot_of_row;
    p.row_of_slot = job.row_of_slot;
    p.offsets = job.offsets;
    p.counts = job.counts;
    p.error = &job.hdr->error;
    int word = 16;
    const bool apart = job.x.base != nullptr && p.num_slots > COUNT_HERE_SLOTS &&
                       job.num_rows * job.row_len * (size_t)row_bytes(job.rows.type) >= APART_BYTES;
    if (!apart && job.x.base != nullptr && job.row_len > 0) {
        const Rows rows[2] = {job.x, job.rows};
        const size_t b = (size_t)row_bytes(job.rows.type);
        word = word_of(rows, 2, job.row_len);
        p.x = static_cast<const unsigned char *>(job.x.base);
        p.rows = static_cast<unsigned char *>(job.rows.base);
        p.x_stride = job.x.stride * b;
        p.rows_stride = job.rows.stride * b;
        p.row_bytes = (uint32_t)(job.row_len * b);
        p.words = (p.row_bytes + unit_bytes(word) - 1) / unit_bytes(word);
    }
    if (apart) {  // the order alone, then a warp for each segment of a row
        const cudaError_t e = launch_tiles<16>(job, p, stream, launches);
        if (e != cudaSuccess) return e;
        ExpertMoveJob move = {};
        move.slot_of_row = job.slot_of_row;
        move.row_of_slot = job.row_of_slot;
        move.num_tokens = job.num_tokens;
        move.num_rows = job.num_rows;
        move.row_len = job.row_len;
        move.top_k = job.top_k;
        move.x = job.x;
        move.rows = job.rows;
        return launch_gather(move, stream, launches);
    }
    if (word == 16) return launch_tiles<16>(job, p, stream, launches);
    if (word == 8) return launch_tiles<8>(job, p, stream, launches);
    if (word == 4) return launch_tiles<4>(job, p, stream, launches);
    return word == 2 ? launch_tiles<2>(job, p, stream, launches) : launch_tiles<ODD_WORD>(job, p, stream, launches);
}

cudaError_t launch_expert_gather(const ExpertMoveJob &job, cudaStream_t stream, int *launches) {
    return launch_gather(job, stream, launches);
}

cudaError_t launch_expert_combine(const ExpertMoveJob &job, cudaStream_t stream, int *launches) {
    return launch_typed(job, false, stream, launches);
}

cudaError_t launch_expert_combine_grad(const ExpertMoveJob &job, cudaStream_t stream, int *launches) {
    return launch_typed(job, true, stream, launches);
}

}  // namespace gbs
