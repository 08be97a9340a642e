// The stable order of token ids by table row, with their positions: what the
// table's gradient sums by.  Keys are the table rows, `vocab` for ids that
// have none (they come last); values are the positions 0 .. n - 1.
//
// Ids are few bits wide and their lists short, so that what counts is the
// number of dependent steps, not the bytes.  Three forms, by length:
//   up to RANK_MOST     every id's place is counted directly,
//                         place(i) = #{j : key_j < key_i} + #{j < i : key_j = key_i},
//                       n^2 comparisons in one launch;
//   then                a counting sort in digits of up to 10 bits (two digits
//                       for any vocabulary below 2^20), up to three launches a
//                       digit;
//   long lists          the library's radix sort.
// Microseconds of the whole gradient with rows of 8 f32 values, random ids below
// 32000 unless said:
//   ids                placed directly   digits   radix
//   2048                      8.4          16.4    36.9
//   4096                     10.2          17.0    38.9
//   8192                     13.4          17.3    34.5
//   9216                     16.0          18.2    39.1
//   9728                     21.4          18.2    40.5   (152 CTAs; some share an SM)
//   131072                                 31.5    43.2
//   196608                                 47.2    43.6
//   196608, below 1000                     38.1    52.6   one digit, two passes
//   196608, below 131072                   35.9    54.5   two digits, three passes
//   524288, below 131072                   50.3    58.8
//   196608, below 2^20                     80.4    55.3   three digits, three passes
//   2^20                                   87.8    67.4
// What bounds the short lists is latency: a launch and a chain of shared-memory
// steps for each of the kernels.
#include "rows.cuh"

namespace gbs {
namespace {

constexpr size_t RANK_MOST = 9216;  // 144 CTAs: one for each of nearly all SMs
constexpr size_t COUNT_MOST = 1 << 17;
constexpr size_t COUNT_MOST_FEWER = 1 << 19;  // where there are fewer digits than radix passes

struct IdParams {
    const void *ids;
    int id_bytes;
    uint32_t n, vocab, inside;  // inside: ids_from(first, vocab)
    int64_t first, padding;
    uint32_t *keys, *vals;  // sorted
    uint32_t *header;       // of the work buffer; cleared by the first kernel
};

template <typename ID> __device__ __forceinline__ uint32_t key_at(const IdParams &p, uint32_t i) {
    return id_key(static_cast<const ID *>(p.ids)[i], p.first, p.padding, p.inside, p.vocab);
}

// The work buffer's header and the words after it that ID_ORDER_CLEARED counts.
__device__ __forceinline__ void clear_header(uint32_t *header) {
    for (uint32_t i = threadIdx.x; i < ID_ORDER_CLEARED / 4; i += blockDim.x) header[i] = 0;
}

// count -= (key < bound), as a subtraction whose borrow the next one takes:
// two instructions a comparison, where a predicate and an add take three.
__device__ __forceinline__ void minus_below(uint32_t &count, uint32_t key, uint32_t bound) {
    asm("{\n\t.reg .u32 rest;\n\tsub.cc.u32 rest, %1, %2;\n\tsubc.u32 %0, %0, 0;\n\t}" : "+r"(count) : "r"(key), "r"(bound));
}

// count += (key < bound) for whole numbers in f32: their difference, held
// between 0 and 1.  Two instructions of a pipe that takes one every cycle, where
// the borrow's are half as fast (8192 ids 13.4 us, 16.2); exact for keys below 2^24.
__device__ __forceinline__ void plus_below(float &count, float key, float bound) {
    float one;
    asm("sub.sat.f32 %0, %1, %2;" : "=f"(one) : "f"(bound), "f"(key));
    count += one;
}

// A CTA places 64 ids, two per lane; its warps share the list in blocks of
// 64, which they read from shared memory (one address for all lanes).  FLOATS:
// keys below 2^24 are compared as numbers in f32.  Bound by the comparisons,
// from 4000 ids on, and before them by reading the list and the launch.
constexpr int RANK_THREADS = 1024;
constexpr int RANK_IDS = 64;
template <bool FLOATS, typename ID> __global__ void __launch_bounds__(RANK_THREADS) id_rank_kernel(const IdParams p) {
    extern __shared__ __align__(16) uint32_t key[];
    __shared__ uint32_t sum[RANK_THREADS / 32][RANK_IDS];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blocks = (p.n + RANK_IDS - 1) / RANK_IDS;
    wait_for_earlier();
    let_next_launch();
    if (blockIdx.x == 0) clear_header(p.header);
    load_keys(key, static_cast<const ID *>(p.ids), p.n, blocks * RANK_IDS, p.first, p.padding, p.inside, p.vocab);
    if (FLOATS)  // in the same order as words, too
        for (uint32_t i = threadIdx.x; i < blocks * RANK_IDS; i += RANK_THREADS) key[i] = __float_as_uint((float)key[i]);
    __syncthreads();
    const uint32_t a = blockIdx.x * RANK_IDS + lane, b = a + 32, ka = key[a], kb = key[b];
    uint32_t ca = 0, cb = 0;
    float fa = 0.0f, fb = 0.0f;
    for (uint32_t block = warp; block < blocks; block += RANK_THREADS / 32) {
        const uint4 *k = reinterpret_cast<const uint4 *>(key + block * RANK_IDS);
        if (block == blockIdx.x) {
            for (uint32_t j = 0; j < RANK_IDS; ++j) {
                const uint32_t kj = key[block * RANK_IDS + j];
                ca -= kj < ka || (kj == ka && j < lane);
                cb -= kj < kb || (kj == kb && j < lane + 32);
            }
        } else if (FLOATS) {  // an equal key counts when its block comes first
            const float equal = block < blockIdx.x ? 1.0f : 0.0f, ta = __uint_as_float(ka) + equal, tb = __uint_as_float(kb) + equal;
            const float4 *f = reinterpret_cast<const float4 *>(k);
#pragma unroll 4
            for (uint32_t j = 0; j < RANK_IDS / 4; ++j) {
                const float4 q = f[j];
                plus_below(fa, q.x, ta);
                plus_below(fb, q.x, tb);
                plus_below(fa, q.y, ta);
                plus_below(fb, q.y, tb);
                plus_below(fa, q.z, ta);
                plus_below(fb, q.z, tb);
                plus_below(fa, q.w, ta);
                plus_below(fb, q.w, tb);
            }
        } else {
            const uint32_t equal = block < blockIdx.x ? 1 : 0, ta = ka + equal, tb = kb + equal;
#pragma unroll 4
            for (uint32_t j = 0; j < RANK_IDS / 4; ++j) {
                const uint4 q = k[j];
                minus_below(ca, q.x, ta);
                minus_below(ca, q.y, ta);
                minus_below(ca, q.z, ta);
                minus_below(ca, q.w, ta);
                minus_below(cb, q.x, tb);
                minus_below(cb, q.y, tb);
                minus_below(cb, q.z, tb);
                minus_below(cb, q.w, tb);
            }
        }
    }
    sum[warp][lane] = (uint32_t)fa - ca;
    sum[warp][lane + 32] = (uint32_t)fb - cb;
    __syncthreads();
    if (threadIdx.x < RANK_IDS) {
        const uint32_t i = blockIdx.x * RANK_IDS + threadIdx.x;
        uint32_t place = 0;
#pragma unroll
        for (int w = 0; w < RANK_THREADS / 32; ++w) place += sum[w][threadIdx.x];
        if (i < p.n) {
            p.keys[place] = FLOATS ? (uint32_t)__uint_as_float(key[i]) : key[i];
            p.vals[place] = i;
        }
    }
}

// One digit of the counting sort: tiles of PLACE_TILE keys.
constexpr int PLACE_THREADS = 256;
constexpr int PLACE_WARPS = PLACE_THREADS / 32;
constexpr uint32_t PLACE_TILE = 1024;
constexpr uint32_t PLACE_ROUNDS = PLACE_TILE / PLACE_THREADS;
constexpr int DIGIT_BITS = 10;  // at most
constexpr uint32_t MOST_PER = (1u << DIGIT_BITS) / PLACE_THREADS;  // digits per thread
constexpr uint32_t SUM_TILES = 32;

struct DigitParams {
    const uint32_t *keys_in, *vals_in;
    uint32_t *keys_out, *vals_out;
    uint32_t *tile_counts, *totals;  // [tiles][bins], [bins]
    uint32_t n, shift, bins;
};

// Counts a tile's digits; the first digit's form also turns ids into keys.
template <bool FIRST, typename ID> __global__ void __launch_bounds__(PLACE_THREADS) id_count_kernel(const IdParams ip, const DigitParams p, uint32_t *keys) {
    __shared__ uint32_t count[1 << DIGIT_BITS];
    for (uint32_t d = threadIdx.x; d < p.bins; d += PLACE_THREADS) count[d] = 0;
    wait_for_earlier();
    let_next_launch();
    if (FIRST && blockIdx.x == 0) clear_header(ip.header);
    __syncthreads();
#pragma unroll
    for (uint32_t r = 0; r < PLACE_ROUNDS; ++r) {
        const uint32_t i = blockIdx.x * PLACE_TILE + r * PLACE_THREADS + threadIdx.x;
        if (i < p.n) {
            const uint32_t k = FIRST ? key_at<ID>(ip, i) : p.keys_in[i];
            if (FIRST) keys[i] = k;
            atomicAdd(&count[(k >> p.shift) & (p.bins - 1)], 1u);
        }
    }
    __syncthreads();
    for (uint32_t d = threadIdx.x; d < p.bins; d += PLACE_THREADS) p.tile_counts[(size_t)blockIdx.x * p.bins + d] = count[d];
}

// Places a tile's keys: a warp takes 128 neighbours, 32 at a time in order,
// so that equal digits keep their order.
// SUM: there are few tiles, and each CTA adds up their counts itself.
template <bool FIRST, bool SUM> __global__ void __launch_bounds__(PLACE_THREADS) id_place_kernel(const DigitParams p) {
    extern __shared__ uint32_t smem[];
    uint32_t *base = smem, *count = base + p.bins;  // count[warp][digit]
    __shared__ uint32_t warp_sum[PLACE_WARPS];
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (uint32_t d = tid; d < PLACE_WARPS * p.bins; d += PLACE_THREADS) count[d] = 0;
    wait_for_earlier();
    let_next_launch();
    // exclusive sum of the digits' totals
    const uint32_t per = (p.bins + PLACE_THREADS - 1) / PLACE_THREADS, d0 = tid * per;
    uint32_t mine = 0, total[MOST_PER], before[MOST_PER];
#pragma unroll
    for (uint32_t k = 0; k < MOST_PER; ++k) {
        const uint32_t d = d0 + k;
        total[k] = before[k] = 0;
        if (k >= per || d >= p.bins) continue;
        if (SUM) {
            const uint32_t tiles = gridDim.x;
#pragma unroll 8
            for (uint32_t t = 0; t < tiles; ++t) {
                const uint32_t c = p.tile_counts[t * p.bins + d];
                total[k] += c;
                if (t < blockIdx.x) before[k] += c;
            }
        } else {
            total[k] = p.totals[d];
            before[k] = p.tile_counts[(size_t)blockIdx.x * p.bins + d];
        }
        mine += total[k];
    }
    uint32_t up = mine;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
        const uint32_t o = __shfl_up_sync(~0u, up, s);
        if (lane >= (uint32_t)s) up += o;
    }
    if (lane == 31) warp_sum[warp] = up;
    __syncthreads();
    up -= mine;
    for (uint32_t w = 0; w < warp; ++w) up += warp_sum[w];
#pragma unroll
    for (uint32_t k = 0; k < MOST_PER; ++k)
        if (k < per && d0 + k < p.bins) {
            base[d0 + k] = up + before[k];
            up += total[k];
        }
    uint32_t key[PLACE_ROUNDS], rank[PLACE_ROUNDS];
    uint32_t *const own = count + warp * p.bins;
    const uint32_t i0 = blockIdx.x * PLACE_TILE + warp * (32 * PLACE_ROUNDS) + lane;
#pragma unroll
    for (uint32_t r = 0; r < PLACE_ROUNDS; ++r) key[r] = i0 + 32 * r < p.n ? p.keys_in[i0 + 32 * r] : ~0u;
#pragma unroll
    for (uint32_t r = 0; r < PLACE_ROUNDS; ++r) {
        const bool on = i0 + 32 * r < p.n;
        const uint32_t d = on ? (key[r] >> p.shift) & (p.bins - 1) : p.bins;
        const uint32_t peers = __match_any_sync(~0u, d), below = __popc(peers & lanemask_lt());
        rank[r] = on ? own[d] + below : 0;
        __syncwarp();
        if (on && below == 0) own[d] += __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    for (uint32_t d = tid; d < p.bins; d += PLACE_THREADS) {
        uint32_t at = base[d];
#pragma unroll
        for (int w = 0; w < PLACE_WARPS; ++w) {
            const uint32_t c = count[w * p.bins + d];
            count[w * p.bins + d] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (uint32_t r = 0; r < PLACE_ROUNDS; ++r) {
        const uint32_t i = i0 + 32 * r;
        if (i < p.n) {
            const uint32_t at = own[(key[r] >> p.shift) & (p.bins - 1)] + rank[r];
            p.keys_out[at] = key[r];
            p.vals_out[at] = FIRST ? i : p.vals_in[i];
        }
    }
}

// Keys and positions for the radix sort.
__global__ void __launch_bounds__(256) id_keys_kernel(const IdParams p, uint32_t *keys, uint32_t *vals) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    if (i >= p.n) return;
    keys[i] = p.id_bytes == 8 ? key_at<int64_t>(p, i) : key_at<int32_t>(p, i);
    vals[i] = i;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

int key_bits(size_t vocab) {
    int bits = 1;
    while ((vocab >> bits) != 0) ++bits;  // the keys are 0 .. vocab
    return bits;
}

// Whether a list too long to be placed directly is sorted by counting.
bool by_digits(size_t n, size_t vocab) {
    const int bits = key_bits(vocab);
    return n <= ((bits + DIGIT_BITS - 1) / DIGIT_BITS < (bits + 7) / 8 ? COUNT_MOST_FEWER : COUNT_MOST);
}

struct Layout {
    size_t keys, vals, keys_alt, vals_alt, hist, base, status, total;
};
Layout layout_of(size_t n, size_t vocab) {
    Layout l = {};
    const size_t list = up256(sizeof(uint32_t) * n);
    size_t off = 0;
    if (n <= RANK_MOST) return l;
    l.keys = off;
    l.vals = off += list;
    off += list;
    if (by_digits(n, vocab)) {
        l.hist = off;  // tile counts and totals
        off += up256(sizeof(uint32_t) * ((n + PLACE_TILE - 1) / PLACE_TILE + 1) << DIGIT_BITS);
    } else {
        const size_t tile = radix_tile_keys(4, 4), hist = up256(sizeof(uint32_t) * MAX_PASSES * 256);
        l.keys_alt = off;
        l.vals_alt = off += list;
        l.hist = off += list;
        l.base = off += hist;
        l.status = off += hist;
        off += up256(status_bytes(n, (n + tile - 1) / tile));
    }
    l.total = off;
    return l;
}

cudaError_t launch_digits(const IdParams &ip, const Layout &l, unsigned char *work, int bits, cudaStream_t stream, int *launches) {
    uint32_t *keys[2] = {reinterpret_cast<uint32_t *>(work + l.keys), ip.keys};
    uint32_t *vals[2] = {reinterpret_cast<uint32_t *>(work + l.vals), ip.vals};
    const int digits = (bits + DIGIT_BITS - 1) / DIGIT_BITS, width = (bits + digits - 1) / digits;
    const uint32_t tiles = (ip.n + PLACE_TILE - 1) / PLACE_TILE;
    cudaError_t e = cudaSuccess;
    // the last digit is placed in the sorted arrays
    const int in = digits % 2 ? 0 : 1;
    for (int d = 0; d < digits; ++d) {
        DigitParams p;
        p.n = ip.n;
        p.shift = (uint32_t)(d * width);
        p.bins = 1u << (bits - d * width < width ? bits - d * width : width);
        p.tile_counts = reinterpret_cast<uint32_t *>(work + l.hist);
        p.totals = p.tile_counts + (size_t)tiles * p.bins;
        p.keys_out = keys[(d + in + 1) % 2];
        p.vals_out = vals[(d + in + 1) % 2];
        p.keys_in = keys[(d + in) % 2];
        p.vals_in = vals[(d + in) % 2];
        uint32_t *const first_keys = keys[in];
        if (d == 0 && ip.id_bytes == 8) e = launch_next(id_count_kernel<true, int64_t>, tiles, PLACE_THREADS, 0, stream, ip, p, first_keys);
        else if (d == 0) e = launch_next(id_count_kernel<true, int32_t>, tiles, PLACE_THREADS, 0, stream, ip, p, first_keys);
        else e = launch_next(id_count_kernel<false, int32_t>, tiles, PLACE_THREADS, 0, stream, ip, p, first_keys);
        if (e != cudaSuccess) return e;
        ++*launches;
        timing_mark(stream);
        const bool sum = tiles <= SUM_TILES;
        if (!sum && (e = launch_tile_scan(p.tile_counts, p.totals, tiles, p.bins, stream, launches)) != cudaSuccess) return e;
        const size_t smem = (1 + PLACE_WARPS) * p.bins * sizeof(uint32_t);
        e = launch_next(sum ? (d == 0 ? id_place_kernel<true, true> : id_place_kernel<false, true>)
                            : (d == 0 ? id_place_kernel<true, false> : id_place_kernel<false, false>),
                        tiles, PLACE_THREADS, smem, stream, p);
        if (e != cudaSuccess) return e;
        ++*launches;
        timing_mark(stream);
    }
    return cudaGetLastError();
}

}  // namespace

size_t id_order_temp_bytes(size_t n, size_t vocab) { return layout_of(n, vocab).total; }

cudaError_t launch_id_order(const IdOrderJob &job, cudaStream_t stream, int *launches) {
    IdParams p = {};
    p.ids = job.ids;
    p.id_bytes = job.id_bytes;
    p.n = (uint32_t)job.n;
    p.vocab = (uint32_t)job.vocab;
    p.inside = (uint32_t)ids_from(job.first_id, job.vocab);
    p.first = job.first_id;
    p.padding = job.padding_id;
    p.keys = job.keys;
    p.vals = job.vals;
    p.header = reinterpret_cast<uint32_t *>(job.hdr);
    const Layout l = layout_of(job.n, job.vocab);
    const int bits = key_bits(job.vocab);
    if (job.n <= RANK_MOST) {
        const uint32_t blocks = (p.n + RANK_IDS - 1) / RANK_IDS;
        const size_t smem = blocks * RANK_IDS * sizeof(uint32_t);
        const bool floats = p.vocab < 1u << 24;
        const auto kernel = p.id_bytes == 8 ? (floats ? id_rank_kernel<true, int64_t> : id_rank_kernel<false, int64_t>)
                                            : (floats ? id_rank_kernel<true, int32_t> : id_rank_kernel<false, int32_t>);
        const cudaError_t e = launch_next(kernel, blocks, RANK_THREADS, smem, stream, p);
        ++*launches;
        timing_mark(stream);
        return e;
    }
    if (by_digits(job.n, job.vocab)) return launch_digits(p, l, job.work, bits, stream, launches);

    cudaError_t e = cudaMemsetAsync(job.hdr, 0, ID_ORDER_CLEARED, stream);
    if (e == cudaSuccess) e = cudaMemsetAsync(job.work + l.hist, 0, sizeof(uint32_t) * MAX_PASSES * 256, stream);
    if (e != cudaSuccess) return e;
    RadixJob r;
    r.kind = KIND_U32;
    r.key_bytes = 4;
    r.val_bytes = 4;
    r.keys_in = job.work + l.keys;
    r.keys_out = job.keys;
    r.keys_alt = job.work + l.keys_alt;
    r.vals_in = job.work + l.vals;
    r.vals_out = job.vals;
    r.vals_alt = job.work + l.vals_alt;
    r.n = job.n;
    r.begin_bit = 0;
    r.end_bit = bits;
    r.num_passes = (bits + 7) / 8;
    r.descending = false;
    r.in_place = false;
    r.hdr = job.hdr;
    r.hist = reinterpret_cast<uint32_t *>(job.work + l.hist);
    r.digit_base = reinterpret_cast<uint32_t *>(job.work + l.base);
    r.status = job.work + l.status;
    r.wide_status = job.n >= WIDE_STATUS_MIN_KEYS;
    r.num_tiles = (uint32_t)((job.n + radix_tile_keys(4, 4) - 1) / radix_tile_keys(4, 4));
    debug_fault_settings(&r.fault_pass, &r.fault_tile, &r.spin_limit);
    id_keys_kernel<<<(p.n + 255) / 256, 256, 0, stream>>>(p, reinterpret_cast<uint32_t *>(job.work + l.keys),
                                                         reinterpret_cast<uint32_t *>(job.work + l.vals));
    ++*launches;
    timing_mark(stream);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_radix_sort(r, stream, launches);
}

}  // namespace gbs
