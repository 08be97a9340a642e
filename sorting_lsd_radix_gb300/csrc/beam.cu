// A beam search's step: the best continuations of a batch's beams, and the
// beams' states moved to where they go on.
//
// select   v[i, w] = score[i] + l[i, w] - log sum_w e^l[i, w] over a batch's beams
//          i and tokens w; the num_out best, best first, ties to the lowest (i, w).
//          Within a beam the order is that of its logits, so a row is read once:
//          a CTA goes through a slice of it by chunks that it holds in registers,
//          adds up the exponentials, and keeps the num_out best logits.  The first
//          chunk's bound is the num_out-th best of 32 groups' maxima; what reaches it
//          (a few more than num_out) is ranked by counting, and the num_out-th best
//          is the bound from then on, made again after 2, 4, 8, ... chunks, so that a
//          logit costs a comparison and only some num_out * log2(chunks) are looked
//          at.  A second kernel merges the slices' lists beam by beam and the beams'
//          by their values, in 64 bits.
//          64 x 8 rows of 131072 bf16: 37 us, the bytes 19.8 at 6787 GB/s.  31 of it
//          are the slices' (343 instructions for 1024 logits of a warp, of which the
//          exponentials are about 100; 512 CTAs on 152 SMs are 3.4 each, so that a
//          sixth of the time some SMs idle), 6 the merge and its launch.  16 x 5 rows of 32000
//          f32 take 8.8, 4 rows of 50257 bf16 7.3 (slices 3).  The sums are formed in
//          32 bits: their logarithms are off by 4e-8 to 8e-8 rms, 2.2e-7 at most, in rows
//          of 32000 to 131072.
// reorder  state[b, j] = state[b, parent[b, j]]: a thread holds the same place of
//          all of a batch's beams, reads what moves before it writes, and leaves
//          alone what stays; in place without a second buffer.  Bound by bytes: 1.5 GB
//          of caches 216 to 230 us, 6.5 to 6.9 TB/s, the rate of a copy.
#include <cfloat>

#include "rows.cuh"

namespace gbs {
namespace {

constexpr uint32_t FULL = 0xFFFFFFFFu;
constexpr int SLICE_THREADS = 256, SLICE_WARPS = SLICE_THREADS / 32;
constexpr uint32_t ROOM = 512;  // keys that a slice keeps at a time
constexpr int JOIN_THREADS = 256, JOIN_WARPS = JOIN_THREADS / 32;
constexpr uint32_t MAX_BEAMS = 32, MOST_SLOTS = MAX_BEAMS * 64;  // the most beams; the most entries of a batch
constexpr uint32_t HEADS = 8;  // a list's entries that are fetched together
constexpr float LOG2E = 1.44269502162933349609375f;  // to 24 bits

__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two values at a time.
__device__ __forceinline__ uint64_t two(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void apart(uint64_t x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ uint64_t fma_two(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_two(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Ordered codes as in the router's choice: larger is better, 0 is minus infinity.
__device__ __forceinline__ uint32_t logit_code(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return x == -INFINITY ? 0u : u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float code_logit(uint32_t c) { return __uint_as_float(c ^ ((uint32_t)(~((int32_t)c >> 31)) | 0x80000000u)); }
__device__ __forceinline__ uint64_t value_code(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return x != x ? ~0ull : x == -INFINITY ? 0ull : u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double code_value(uint64_t c) {
    return c == 0 ? -INFINITY : __longlong_as_double((long long)(c ^ ((uint64_t)(~((int64_t)c >> 63)) | 0x8000000000000000ull)));
}

// A slice's largest logit and the sum of e^(x - top).
struct Stat {
    float top, sum;
};
// What such a sum by `top` is multiplied with to be one by `to`, the larger.
__device__ __forceinline__ float rescale(float top, float to) { return top == -INFINITY ? 0.0f : exp2_of((top - to) * LOG2E); }

// A thread's sum on the way is kept by a base: sum * 2^base(top), so that e^x is one
// multiply-add and 2^x.  The base is off from the largest logit's exponent by up to
// 2^-24 of itself, so from 2^20 on, where that would begin to count (0.09; 2^120 at
// 2e9), it is a sum of e^(x - top) already.
__device__ __forceinline__ bool is_far(float top) { return !(fabsf(top) < 1048576.0f); }
__device__ __forceinline__ float base_of(float top) { return __fmul_rn(top, LOG2E); }
// What a sum on the way by `top` is multiplied with to be one by `to`, the larger.
__device__ __forceinline__ float rescale_base(float top, float to) {
    if (is_far(to)) return is_far(top) ? rescale(top, to) : exp2_of(fmaf(-to, LOG2E, base_of(top)));
    return exp2_of(is_far(top) ? fmaf(top, LOG2E, -base_of(to)) : base_of(top) - base_of(to));
}

struct SelectParams {
    const void *logits;
    size_t stride;
    uint32_t rows, vocab, slices, chunks, num_out;  // a slice is so many chunks of a row
    uint32_t beams;
    const float *scores;
    const uint8_t *finished;  // nullptr: none
    int32_t end_id;
    uint64_t *lists;  // [rows][slices][num_out]: the best logits' codes over ~token, best first, 0 for none
    Stat *stats;      // [rows][slices]
    float *scores_out;
    int32_t *beams_out, *tokens_out;
    uint32_t *error;
};

// Whether a beam exists and goes on.
__device__ __forceinline__ bool is_open(const SelectParams &p, uint32_t row) {
    return p.scores[row] != -INFINITY && !(p.finished && p.finished[row]);
}

// A pack of a row that is read once (kept out of L1: 512 rows of 131072 bf16
// 39.3 -> 38.2 us).
template <typename T> __device__ __forceinline__ Pack<T, 16 / sizeof(T)> load_streamed(const T *p) {
    Pack<T, 16 / sizeof(T)> x;
    uint32_t *w = reinterpret_cast<uint32_t *>(&x);
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
    return x;
}

// The largest of a pack's values, NaN left out where there is another.
template <int P> __device__ __forceinline__ float max_of(const Pack<float, P> &a) {
    float m = a.v[0];
#pragma unroll
    for (int j = 1; j < P; ++j) m = fmaxf(m, a.v[j]);
    return m;
}
__device__ __forceinline__ float max_of(const Pack<__half, 8> &a) {
    const __half2 *h = reinterpret_cast<const __half2 *>(&a);
    const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float max_of(const Pack<__nv_bfloat16, 8> &a) {
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&a);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
}

__device__ __forceinline__ uint64_t key_of(float x, uint32_t token) { return (uint64_t)logit_code(x) << 32 | (uint32_t)~token; }

// The num_out best of the n keys in `from`, in order, to `to`; a CTA's work, a
// key's comparisons shared by four lanes.
__device__ __forceinline__ void rank_keys(const uint64_t *from, uint32_t n, uint64_t *to, uint32_t num_out) {
    const uint32_t sub = threadIdx.x & 3;
    for (uint32_t i0 = 0; i0 < n; i0 += SLICE_THREADS / 4) {
        const uint32_t i = i0 + threadIdx.x / 4;
        const uint64_t key = i < n ? from[i] : ~0ull;
        uint32_t rank = 0;
#pragma unroll 4
        for (uint32_t k = sub; k < n; k += 4) rank += from[k] > key;
        rank += __shfl_xor_sync(FULL, rank, 1);
        rank += __shfl_xor_sync(FULL, rank, 2);
        if (sub == 0 && i < n && rank < num_out) to[rank] = key;
    }
}

// The next larger value of 32 bits, of minus infinity the lowest; infinity itself.
__device__ __forceinline__ float above(float x) { return fabsf(x) == INFINITY ? fmaxf(x, -FLT_MAX) : code_logit(logit_code(x) + 1); }

// A slice of a row: PACKS packs of 16 bytes a thread at a time.
template <typename T, int PACKS, bool ODD> __global__ void __launch_bounds__(SLICE_THREADS, 4) beam_slice_kernel(const SelectParams p) {
    constexpr int P = 16 / (int)sizeof(T);
    constexpr uint32_t CHUNK = SLICE_THREADS * PACKS * P;
    __shared__ uint64_t found[2][ROOM];
    __shared__ float tops[SLICE_WARPS][32], warp_top[SLICE_WARPS], warp_sum[SLICE_WARPS];
    __shared__ uint32_t count, totals[3];
    wait_for_earlier();
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blockIdx.x == 0 && tid == 0) *p.error = 0;
    const uint32_t row = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
    const T *logits = static_cast<const T *>(p.logits) + (size_t)row * p.stride;
    const uint32_t first = slice * p.chunks * CHUNK, end = min(p.vocab - first, p.chunks * CHUNK);  // end: values of the slice
    if (tid == 0) count = totals[0] = totals[1] = totals[2] = 0;

    Pack<T, P> x[PACKS];
    auto load = [&](uint32_t at) {
        const T *from = logits + first + at + tid * P;
        if (!ODD && at + CHUNK <= end) {
#pragma unroll
            for (int i = 0; i < PACKS; ++i) x[i] = load_streamed(from + i * SLICE_THREADS * P);
        } else {
#pragma unroll
            for (int i = 0; i < PACKS; ++i) {
                const uint32_t c = at + (i * SLICE_THREADS + tid) * P;
                x[i] = load_row<ODD, T>(logits, first + c, p.vocab, c < end);
#pragma unroll
                for (int j = 0; j < P; ++j)
                    if (c + j >= end) x[i].v[j] = from_f32<T>(-INFINITY);
            }
        }
    };
    auto value_at = [&](uint32_t token) {
        const float v = to_f32(logits[token]);
        return v != v ? INFINITY : v;
    };
    // a finished beam's row may have nothing behind it; other rows' logits are on their way while the score is looked at
    // (16 x 5 rows of 32000 with flags 9.3 us either way; with the scores before the logits too 10.7, 4 rows of 50257
    // 10.2 instead of 7.9)
    if (p.finished && p.finished[row]) return;
    load(0);
    if (p.scores[row] == -INFINITY) return;
    float top = -INFINITY, sum = 0.0f;
    float bound = 0.0f;  // what a logit has to reach: num_out of those before do, or are just below
    uint32_t which = 0;  // the half of found that is in use
    uint32_t since = 0;  // what was looked at since the keys were cut
    for (uint32_t at = 0; at < end; at += CHUNK) {
        const bool last = at + CHUNK >= end;
        // the chunk after next into L2 (512 rows of 131072 bf16 44.0 -> 42.1 us)
        if (!ODD && tid == 0 && at + 3 * CHUNK <= end) prefetch_l2_bulk(logits + first + at + 2 * CHUNK, CHUNK * (uint32_t)sizeof(T));
        float most[PACKS], high = -INFINITY;
#pragma unroll
        for (int i = 0; i < PACKS; ++i) {
            most[i] = max_of(x[i]);
            high = fmaxf(high, most[i]);
        }
        const float before = top;
        top = fmaxf(top, high);
        if (is_far(top)) {
            if (top != -INFINITY) {
                sum *= rescale_base(before, top);
#pragma unroll
                for (int i = 0; i < PACKS; ++i)
#pragma unroll
                    for (int j = 0; j < P; ++j) sum += exp2_of((to_f32(x[i].v[j]) - top) * LOG2E);
            } else {  // nothing but masked logits, or NaN
#pragma unroll
                for (int i = 0; i < PACKS; ++i)
#pragma unroll
                    for (int j = 0; j < P; ++j) sum += to_f32(x[i].v[j]) == -INFINITY ? 0.0f : NAN;
            }
        } else {
            const float base = base_of(top);
            sum *= rescale_base(before, top);
            uint64_t part = 0;
            const uint64_t by = two(LOG2E, LOG2E), less = two(-base, -base);
#pragma unroll
            for (int i = 0; i < PACKS; ++i)
#pragma unroll
                for (int j = 0; j < P; j += 2) {
                    float a, b;
                    apart(fma_two(two(to_f32(x[i].v[j]), to_f32(x[i].v[j + 1])), by, less), a, b);
                    part = add_two(part, two(exp2_of(a), exp2_of(b)));
                }
            float a, b;
            apart(part, a, b);
            sum += a + b;
        }
        if (sum != sum) {  // NaN, or an infinity: the beam's values are NaN, its NaN logits come first
            top = high = INFINITY;
#pragma unroll
            for (int i = 0; i < PACKS; ++i) most[i] = INFINITY;
        }
        if (at == 0) {
            // the num_out-th best of 32 groups' maxima (from 33 on the least of 64): that many logits reach it.  A group
            // is a lane's threads of all warps (of every other one), so that a short slice leaves few empty
            tops[warp][lane] = high;
            __syncthreads();
            float even = tops[0][lane], odd = tops[1][lane];
#pragma unroll
            for (int w = 2; w < SLICE_WARPS; w += 2) even = fmaxf(even, tops[w][lane]), odd = fmaxf(odd, tops[w + 1][lane]);
            bound = fminf(even, odd);
            if (p.num_out <= 32) {
                const float mine = fmaxf(even, odd);
                uint32_t better = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) better += __shfl_sync(FULL, mine, i) > mine;
                bound = better < p.num_out ? mine : INFINITY;
            }
#pragma unroll
            for (int d = 16; d > 0; d /= 2) bound = fminf(bound, __shfl_xor_sync(FULL, bound, d));
            bound = fmaxf(bound, -FLT_MAX);
        }
        uint32_t hits = 0;
        float value = 0.0f;  // of the last hit
        if (high >= bound) {
#pragma unroll
            for (int i = 0; i < PACKS; ++i)
                if (most[i] >= bound)
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        const float v = to_f32(x[i].v[j]);
                        if (!(v < bound)) hits |= 1u << (i * P + j), value = v;
                    }
        }
        if (!last) load(at + CHUNK);
        while (hits) {
            const uint32_t h = 31 - __clz(hits), token = first + at + ((h / P) * SLICE_THREADS + tid) * P + h % P;
            hits ^= 1u << h;
            const uint32_t to = atomicAdd(&count, 1u);
            if (to < ROOM) found[which][to] = key_of(value != value ? INFINITY : value, token);
            if (hits) {  // a thread's others are read again
                const uint32_t g = 31 - __clz(hits);
                value = to_f32(logits[first + at + ((g / P) * SLICE_THREADS + tid) * P + g % P]);
            }
        }
        // cut to num_out after 1, 2, 4, ... chunks: each time about num_out more have reached the bound
        const uint32_t done = at / CHUNK + 1;
        if ((done & (done - 1)) != 0 && !last) continue;
        __syncthreads();
        uint32_t n = count;
        if (n > ROOM) {
            // rows that mislead the bound, or too many equals: the num_out-th best key of what was looked at since the
            // last cut, and of what was kept then, bit by bit
            uint64_t least = 0;
            const uint32_t stop = first + min(at + CHUNK, end);
            auto old = [&](uint64_t key) { return ~(uint32_t)key < first + since; };
            for (int b = 63; b >= 0; --b) {
                const uint64_t up = least | 1ull << b;
                uint32_t mine = 0;
                for (uint32_t t = first + since + tid; t < stop; t += SLICE_THREADS) {
                    const float v = value_at(t);
                    mine += v != -INFINITY && key_of(v, t) >= up;
                }
                for (uint32_t k = tid; k < ROOM; k += SLICE_THREADS) mine += old(found[which][k]) && found[which][k] >= up;
                mine = __reduce_add_sync(FULL, mine);
                // three counters by turns: the one cleared here is added to after the next barrier
                if (lane == 0 && mine) atomicAdd(&totals[b % 3], mine);
                __syncthreads();
                if (totals[b % 3] >= p.num_out) least = up;
                if (tid == 0) totals[(b + 1) % 3] = 0;
            }
            if (tid == 0) count = 0;
            __syncthreads();
            if (tid == 0) totals[0] = 0;
            for (uint32_t t = first + since + tid; t < stop; t += SLICE_THREADS) {
                const float v = value_at(t);
                if (v != -INFINITY && key_of(v, t) >= least) found[which ^ 1][atomicAdd(&count, 1u)] = key_of(v, t);
            }
            for (uint32_t k = tid; k < ROOM; k += SLICE_THREADS) {
                const uint64_t key = found[which][k];
                if (old(key) && key >= least) found[which ^ 1][atomicAdd(&count, 1u)] = key;
            }
            __syncthreads();
            n = count;
            which ^= 1;
        }
        if (last) {
            uint64_t *list = p.lists + (size_t)blockIdx.x * p.num_out;
            rank_keys(found[which], n, list, p.num_out);
            for (uint32_t i = n + tid; i < p.num_out; i += SLICE_THREADS) list[i] = 0;
        } else {
            rank_keys(found[which], n, found[which ^ 1], p.num_out);
            __syncthreads();
            which ^= 1;
            if (tid == 0) count = min(n, p.num_out);
            // a later equal does not count, its token is higher
            bound = n >= p.num_out ? above(code_logit((uint32_t)(found[which][p.num_out - 1] >> 32))) : -FLT_MAX;
            since = at + CHUNK;
            __syncthreads();
        }
    }
    if (!is_far(top)) sum *= exp2_of(fmaf(-top, LOG2E, base_of(top)));
    float all = top;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) all = fmaxf(all, __shfl_xor_sync(FULL, all, d));
    sum = top == -INFINITY ? 0.0f : sum * rescale(top, all);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(FULL, sum, d);
    if (lane == 0) warp_top[warp] = all, warp_sum[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        float t = warp_top[0], s = 0.0f;
        for (int w = 1; w < SLICE_WARPS; ++w) t = fmaxf(t, warp_top[w]);
        for (int w = 0; w < SLICE_WARPS; ++w) s += warp_sum[w] * rescale(warp_top[w], t);
        p.stats[blockIdx.x] = {t, s};
    }
}

// -log r for r = round(256 / (1 + (i + 0.5) / 32)) / 256.
__device__ const double MINUS_LOG[32] = {
    0.015748356968139168, 0.043919233934835489, 0.077117303344431287, 0.10275973395776894,
    0.13353139262452263, 0.16068238169047347, 0.18388527877013736, 0.21245865121419341,
    0.23690974707835771, 0.26197371574157396, 0.28248725557467691, 0.30873548164961329,
    0.33024168687057687, 0.35222059358935209, 0.3746934494414107, 0.39768296766610944,
    0.41527872955648898, 0.43923197057898189, 0.45758110924717837, 0.47627324225933093,
    0.49532143723002542, 0.514739523087127, 0.53454215038330677, 0.54796517071544737,
    0.56844370205898809, 0.58935038687830177, 0.6035350218702582, 0.61792375932235777,
    0.63990266604113299, 0.65482831625780868, 0.66998012127841089, 0.68536504011789035,
};

// One CTA for a batch.  A warp makes a beam's sum and merges the lists of its
// slices while one more takes the sums' logarithms; then the beams' entries are
// ranked against one another by counting.  64-bit instructions are slow here (a
// call of log is a chain of about 1.2 us), so a sum's logarithm is made of few:
//   log(2^e m) = e log 2 - log r + log(1 + u),  u = m r - 1,  |u| < 1 / 50,
// with r of 9 bits the inverse of m's interval of 32, and the terms from u^2 on in
// 32 bits, for which they are small enough (all in all off by 3e-11).
__global__ void __launch_bounds__(JOIN_THREADS + 32) beam_join_kernel(const SelectParams p) {
    extern __shared__ __align__(16) unsigned char shared[];
    __shared__ uint64_t heads[JOIN_WARPS][32][HEADS + 1];
    __shared__ double over[MAX_BEAMS];
    __shared__ float tops[MAX_BEAMS], sums[MAX_BEAMS][2];
    __shared__ uint32_t open[MAX_BEAMS], all;
    wait_for_earlier();
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = p.num_out, slots = p.beams * k;
    uint64_t *value = reinterpret_cast<uint64_t *>(shared);  // [beams][k] the logits' codes, then the values', 0 for none
    uint64_t *merged = value + slots;                        // [warps][2][k]
    int32_t *token = reinterpret_cast<int32_t *>(merged + JOIN_WARPS * 2 * k);  // [beams][k]
    float *rounded = reinterpret_cast<float *>(token + slots);                  // [beams][k] the values
    const uint32_t row0 = blockIdx.x * p.beams;
    if (tid == 0) all = 0;
    const double minus_log = warp == JOIN_WARPS ? MINUS_LOG[lane] : 0.0;
    // the slices' lists 31 at a time, by lanes from 1 on
    auto list_of = [&](uint32_t row, uint32_t s0) { return p.lists + ((size_t)row * p.slices + s0 + lane - 1) * k; };
    auto fetch = [&](uint32_t row, uint32_t s0) {
        const bool mine = lane > 0 && s0 + lane - 1 < p.slices;
        const uint32_t *list = reinterpret_cast<const uint32_t *>(list_of(row, s0));
        Pack<uint32_t, 2> entry[HEADS];  // all on their way at once
#pragma unroll
        for (uint32_t j = 0; j < HEADS; ++j) entry[j] = load_pack_if<uint32_t, 2>(list + 2 * j, mine && j < k);
#pragma unroll
        for (uint32_t j = 0; j < HEADS; ++j)
            if (mine) heads[warp][lane][j] = (uint64_t)entry[j].v[1] << 32 | entry[j].v[0];
    };
    if (warp < JOIN_WARPS) {
        if (warp < p.beams && p.slices > 1) fetch(row0 + warp, 0);  // on its way
        for (uint32_t i = warp; i < p.beams; i += JOIN_WARPS) {
            const uint32_t row = row0 + i;
            const Stat *stat = p.stats + (size_t)row * p.slices;
            const Stat own = lane < p.slices ? stat[lane] : Stat{-INFINITY, 0.0f};
            const bool goes_on = is_open(p, row);
            if (lane == 0) open[i] = goes_on;
            if (!goes_on) continue;
            float top = own.top;
            for (uint32_t s = lane + 32; s < p.slices; s += 32) top = fmaxf(top, stat[s].top);
#pragma unroll
            for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(FULL, top, d));
            // the sum and what its roundings lost
            float sum = own.sum * rescale(own.top, top), lost = 0.0f;
            auto add = [&](float x) {
                const float s = sum + x, part = s - sum;
                lost += (sum - (s - part)) + (x - part);
                sum = s;
            };
            for (uint32_t s = lane + 32; s < p.slices; s += 32) add(stat[s].sum * rescale(stat[s].top, top));
            for (uint32_t d = 1; d < 32 && d < p.slices; d *= 2) {
                const float x = __shfl_xor_sync(FULL, sum, d);
                lost += __shfl_xor_sync(FULL, lost, d);
                add(x);
            }
            if (lane == 0) tops[i] = top, sums[i][0] = sum, sums[i][1] = lost;
        }
    }
    __syncthreads();
    if (warp < JOIN_WARPS) {
        for (uint32_t i = warp; i < p.beams; i += JOIN_WARPS) {
            const uint32_t row = row0 + i;
            if (!open[i]) {
                const float score = p.scores[row];
                const bool ended = score != -INFINITY;
                for (uint32_t r = lane; r < k; r += 32) value[i * k + r] = r == 0 && ended ? value_code((double)score) : 0;
                if (lane == 0) {
                    token[i * k] = p.end_id;
                    if (ended) atomicAdd(&all, 1u);
                }
                continue;
            }
            // lane 0 has what was merged before: lower lanes have lower tokens, so the lowest of equals comes first
            uint64_t *from = merged + warp * 2 * k, *to = from + k;
            uint32_t have = 0;
            if (p.slices == 1) {  // in order already
                for (uint32_t r = lane; r < k; r += 32) to[r] = p.lists[(size_t)row * k + r];
                __syncwarp();
                for (uint32_t r0 = 0; r0 < k; r0 += 32) have += __popc(__ballot_sync(FULL, r0 + lane < k && to[r0 + lane] != 0));
                from = to;
            }
            for (uint32_t s0 = 0; s0 < p.slices && p.slices > 1; s0 += 31) {
                const bool mine = lane > 0 && s0 + lane - 1 < p.slices;
                const uint64_t *list = list_of(row, mine ? s0 : 0);
                const uint32_t length = lane == 0 ? have : mine ? k : 0;
                if (s0 > 0 || i != warp) fetch(row, s0);
                __syncwarp();
                auto entry = [&](uint32_t at) { return at >= length ? 0ull : lane == 0 ? from[at] : at < HEADS ? heads[warp][lane][at] : list[at]; };
                uint64_t head = entry(0), next = entry(1);
                uint32_t at = 2, r = 0;
                for (; r < k; ++r) {
                    const uint32_t code = (uint32_t)(head >> 32), best = __reduce_max_sync(FULL, code);
                    if (best == 0) break;
                    const uint32_t equal = __ballot_sync(FULL, code == best);
                    if (code == best && (equal & lanemask_lt()) == 0) {
                        to[r] = head;
                        head = next;
                        next = entry(at++);
                    }
                }
                __syncwarp();
                have = r;
                uint64_t *other = from;
                from = to;
                to = other;
            }
            for (uint32_t r = lane; r < k; r += 32) {
                value[i * k + r] = r < have ? from[r] >> 32 : 0;
                token[i * k + r] = r < have ? (int32_t)~(uint32_t)from[r] : -1;
            }
            if (lane == 0) atomicAdd(&all, have);
            __syncwarp();
        }
    } else {
        const bool mine = lane < p.beams && open[lane];
        const double sum = mine ? (double)sums[lane][0] + (double)sums[lane][1] : 1.0;
        const uint64_t bits = (uint64_t)__double_as_longlong(sum);
        const uint32_t at = (uint32_t)(bits >> 47) & 31;  // m's interval
        const double t = __shfl_sync(FULL, minus_log, at);
        const float r = rintf(256.0f / (1.0f + ((float)at + 0.5f) / 32.0f)) / 256.0f;
        const double m = __longlong_as_double((long long)((bits & 0x000fffffffffffffull) | 0x3ff0000000000000ull));
        const double u = m * (double)r - 1.0, ln2 = 0.693147180559945309417;
        const float v = (float)u, series = v * v * (-0.5f + v * (1.0f / 3 + v * (-0.25f + v * (0.2f - v * (1.0f / 6)))));
        double l = (double)((int)(bits >> 52) - 1023) * ln2 + (t + (u + (double)series));
        if (!(sum > 0.0 && sum < INFINITY)) l = log(sum);
        if (mine) over[lane] = l;
    }
    __syncthreads();
    for (uint32_t q = tid; q < slots; q += JOIN_THREADS + 32) {
        const uint32_t i = q / k;
        uint64_t v = value[q];
        if (v == 0) continue;
        if (open[i]) v = value_code((double)p.scores[row0 + i] + (((double)code_logit((uint32_t)v) - (double)tops[i]) - over[i]));
        rounded[q] = (float)code_value(v);
        // the place in the last bits, 2^-42 of the value: no two are equal, and equals come by beam and place
        value[q] = (v & ~(uint64_t)(MOST_SLOTS - 1)) | (MOST_SLOTS - 1 - q);
    }
    __syncthreads();
    // an entry's rank by counting, shared by several lanes where there are few
    const uint32_t share = slots <= 32 ? 8 : slots <= 64 ? 4 : slots <= 128 ? 2 : 1, sub = tid & (share - 1);
    const size_t out = (size_t)blockIdx.x * k;
    if (warp < JOIN_WARPS) {
        for (uint32_t q0 = 0; q0 < slots; q0 += JOIN_THREADS / share) {
            const uint32_t q = q0 + tid / share;
            const uint64_t v = q < slots ? value[q] : 0;
            uint32_t rank = 0;
#pragma unroll 8
            for (uint32_t o = sub; o < slots; o += share) rank += value[o] > v;
            for (uint32_t d = 1; d < share; d *= 2) rank += __shfl_xor_sync(FULL, rank, d);
            if (sub == 0 && v != 0 && rank < k) {
                p.scores_out[out + rank] = rounded[q];
                p.beams_out[out + rank] = (int32_t)(q / k);
                p.tokens_out[out + rank] = token[q];
            }
        }
    }
    for (uint32_t r = all + tid; r < k; r += JOIN_THREADS + 32) {
        p.scores_out[out + r] = -INFINITY;
        p.beams_out[out + r] = -1;
        p.tokens_out[out + r] = -1;
    }
}

// How rows are cut: chunks of 64 bytes a thread, in slices enough for SLICES CTAs
// where there are as many chunks (512 rows of 131072 bf16: whole rows 38 us, two
// slices a row 41, three 47: each begins without a bound); or, with fewer chunks
// than SMs, of 16 bytes (32 for f32), each a slice.
constexpr size_t SLICES = 152 * 3;
struct Cut {
    uint32_t chunk, chunks, slices;
    bool small;
};
Cut cut_of(size_t rows, size_t vocab, int type) {
    const size_t value = row_bytes(type), wide = SLICE_THREADS * 64 / value;
    size_t count = (vocab + wide - 1) / wide;
    if (rows * count < 152) {
        const size_t narrow = SLICE_THREADS * 8;
        return {(uint32_t)narrow, 1, (uint32_t)((vocab + narrow - 1) / narrow), true};
    }
    size_t chunks = rows * count / SLICES;
    chunks = chunks < 1 ? 1 : chunks > count ? count : chunks;
    const size_t slices = (count + chunks - 1) / chunks;
    return {(uint32_t)wide, (uint32_t)((count + slices - 1) / slices), (uint32_t)slices, false};
}

template <typename T> cudaError_t launch_slices(const SelectParams &p, const Cut &cut, bool odd, cudaStream_t stream) {
    const dim3 grid(p.rows * p.slices), block(SLICE_THREADS);
    constexpr int FEW = sizeof(T) == 4 ? 2 : 1;
    if (!cut.small) return launch_next(odd ? beam_slice_kernel<T, 4, true> : beam_slice_kernel<T, 4, false>, grid, block, 0, stream, p);
    return launch_next(odd ? beam_slice_kernel<T, FEW, true> : beam_slice_kernel<T, FEW, false>, grid, block, 0, stream, p);
}

// ---------------------------------------------------------------------------
// Reordering
// ---------------------------------------------------------------------------

// Division by a number that a launch keeps (Granlund and Montgomery, 1994).
struct Divisor {
    uint32_t d, m, s1, s2;
    Divisor(uint32_t by = 1) : d(by) {
        uint32_t l = 0;
        while (l < 32 && ((uint64_t)1 << l) < by) ++l;
        m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << l) - by)) / by + 1);
        s1 = l < 1 ? l : 1;
        s2 = l < 1 ? 0 : l - 1;
    }
    __device__ __forceinline__ uint32_t of(uint32_t n) const {
        const uint32_t t = __umulhi(m, n);
        return (t + ((n - t) >> s1)) >> s2;
    }
};

struct ReorderParams {
    const unsigned char *in;
    unsigned char *out;
    const int32_t *parents;  // [batch][into]
    uint32_t beams, into, total;  // total: places of outer * batch * segments * units
    Divisor unit, segment, batch;  // units of a segment, segments, batches
    uint32_t rest;                 // bytes of a segment's last unit, 0: a whole one
    size_t in_outer, in_batch, in_beam, in_segment, out_outer, out_batch, out_beam, out_segment;  // bytes
    int place;
};

// A unit where `on`, one predicated instruction: with a branch around each load
// they wait for one another (476 us instead of 219 for 1.5 GB of caches).
template <typename W> __device__ __forceinline__ W load_unit(const unsigned char *p, bool on) {
    if constexpr (sizeof(W) == 16) {
        const Pack<uint32_t, 4> x = load_pack_if<uint32_t, 4>(reinterpret_cast<const uint32_t *>(p), on);
        return make_uint4(x.v[0], x.v[1], x.v[2], x.v[3]);
    } else if constexpr (sizeof(W) == 8) {
        const Pack<uint32_t, 2> x = load_pack_if<uint32_t, 2>(reinterpret_cast<const uint32_t *>(p), on);
        return (W)x.v[1] << 32 | x.v[0];
    } else if constexpr (sizeof(W) == 4) {
        return load_pack_if<uint32_t, 1>(reinterpret_cast<const uint32_t *>(p), on).v[0];
    } else {
        uint32_t x = 0;
        if constexpr (sizeof(W) == 2)
            asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q ld.global.u16 %0, [%1];\n\t}" : "+r"(x) : "l"(p), "r"((uint32_t)on));
        else
            asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q ld.global.u8 %0, [%1];\n\t}" : "+r"(x) : "l"(p), "r"((uint32_t)on));
        return (W)x;
    }
}

// B: the most beams; W: words of a unit's bytes; U: units of a thread; REST:
// segments may end inside a unit.
template <int B, typename W, int U, int THREADS, bool REST> __global__ void __launch_bounds__(THREADS) beam_reorder_kernel(const ReorderParams p) {
    wait_for_earlier();
    uint32_t at[U];
    const unsigned char *from[U];
    unsigned char *to[U];
    const int32_t *parents[U];
    W v[U][B];
    uint32_t moved[U];
    bool whole[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        at[i] = (blockIdx.x * U + i) * THREADS + threadIdx.x;
        const uint32_t n = min(at[i], p.total - 1);
        const uint32_t segs = p.unit.of(n), unit = n - segs * p.unit.d;
        const uint32_t rows = p.segment.of(segs), seg = segs - rows * p.segment.d;
        const uint32_t outer = p.batch.of(rows), b = rows - outer * p.batch.d;
        from[i] = p.in + outer * p.in_outer + b * p.in_batch + seg * p.in_segment + (size_t)unit * sizeof(W);
        to[i] = p.out + outer * p.out_outer + b * p.out_batch + seg * p.out_segment + (size_t)unit * sizeof(W);
        parents[i] = p.parents + (size_t)b * p.into;
        moved[i] = 0;
        whole[i] = !REST || unit + 1 < p.unit.d;
    }
    auto parent_of = [&](int i, int j) {  // 32 bits without sign: none where it is not below p.beams, nor where nothing moves
        if ((uint32_t)j >= p.into || at[i] >= p.total) return FULL;
        const uint32_t parent = (uint32_t)parents[i][j];
        return p.place && parent == (uint32_t)j ? FULL : parent;
    };
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const uint32_t parent = parent_of(i, j);
            const bool on = parent < p.beams && whole[i];
            v[i][j] = load_unit<W>(from[i] + (on ? parent * p.in_beam : 0), on);
            moved[i] |= (uint32_t)on << j;
        }
    asm volatile("" ::: "memory");  // in place: what moves is read before any of it is written
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < B; ++j)
            if ((moved[i] >> j) & 1) *reinterpret_cast<W *>(to[i] + j * p.out_beam) = v[i][j];
    if constexpr (REST) {  // a segment's end, byte by byte
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (whole[i]) continue;
            for (uint32_t k = 0; k < p.rest; ++k) {
                uint8_t b[B];
#pragma unroll
                for (int j = 0; j < B; ++j) {
                    const uint32_t parent = parent_of(i, j);
                    if (parent < p.beams) b[j] = from[i][parent * p.in_beam + k];
                }
#pragma unroll
                for (int j = 0; j < B; ++j)
                    if (parent_of(i, j) < p.beams) to[i][j * p.out_beam + k] = b[j];
            }
        }
    }
}

template <int B, typename W, int U, int THREADS> cudaError_t launch_reorder_as(const ReorderParams &p, cudaStream_t stream) {
    constexpr uint32_t EACH = THREADS * U;
    return launch_next(p.rest ? beam_reorder_kernel<B, W, U, THREADS, sizeof(W) != 1> : beam_reorder_kernel<B, W, U, THREADS, false>,
                       dim3((p.total + EACH - 1) / EACH), dim3(THREADS), 0, stream, p);
}
// Few beams take several units a thread, for as many loads on their way (two
// beams, 250 MB: one unit 51 us, two 41, four 39); 32 beams' values are many
// registers, and CTAs of 128 threads leave more room (161 -> 134 us for 0.8 GB).
template <typename W> cudaError_t launch_reorder_by(const ReorderParams &p, cudaStream_t stream) {
    if (p.into <= 2) return launch_reorder_as<2, W, 4, 256>(p, stream);
    if (p.into <= 4) return launch_reorder_as<4, W, 2, 256>(p, stream);
    if (p.into <= 8) return launch_reorder_as<8, W, 1, 256>(p, stream);
    if (p.into <= 16) return launch_reorder_as<16, W, 1, 256>(p, stream);
    return launch_reorder_as<32, W, 1, 128>(p, stream);
}

}  // namespace

// The work buffer: header, statistics, lists.
static size_t stats_bytes(size_t rows, size_t slices) { return (rows * slices * sizeof(Stat) + 255) / 256 * 256; }
size_t beam_slices(size_t rows, size_t vocab, int type) { return cut_of(rows, vocab, type).slices; }
size_t beam_select_temp_bytes(size_t rows, size_t vocab, int type, size_t num_out) {
    const size_t slices = beam_slices(rows, vocab, type);
    return sizeof(Header) + stats_bytes(rows, slices) + rows * slices * num_out * sizeof(uint64_t);
}

cudaError_t launch_beam_select(const BeamSelectJob &job, cudaStream_t stream, int *launches) {
    const size_t rows = job.batch * job.beams;
    // no beam: the work buffer still says that nothing went wrong
    if (rows == 0) return cudaMemsetAsync(job.temp, 0, sizeof(Header), stream);
    SelectParams p = {};
    p.logits = job.logits.base;
    p.stride = job.logits.stride;
    p.rows = (uint32_t)rows;
    p.vocab = (uint32_t)job.vocab;
    const Cut cut = cut_of(rows, job.vocab, job.logits.type);
    p.slices = cut.slices;
    p.chunks = cut.chunks;
    p.num_out = job.num_out;
    p.beams = job.beams;
    p.scores = job.scores;
    p.finished = job.finished;
    p.end_id = job.end_id;
    p.error = &reinterpret_cast<Header *>(job.temp)->error;
    p.stats = reinterpret_cast<Stat *>(job.temp + sizeof(Header));
    p.lists = reinterpret_cast<uint64_t *>(job.temp + sizeof(Header) + stats_bytes(rows, p.slices));
    p.scores_out = job.scores_out;
    p.beams_out = job.beams_out;
    p.tokens_out = job.tokens_out;
    const bool odd = !whole_packs(&job.logits, 1, job.vocab);
    cudaError_t e = job.logits.type == ROW_F32   ? launch_slices<float>(p, cut, odd, stream)
                    : job.logits.type == ROW_F16 ? launch_slices<__half>(p, cut, odd, stream)
                                                 : launch_slices<__nv_bfloat16>(p, cut, odd, stream);
    if (e != cudaSuccess) return e;
    ++*launches;
    timing_mark(stream);
    const size_t room = (size_t)p.beams * p.num_out * 16 + JOIN_WARPS * 2 * (size_t)p.num_out * 8;
    static PerDeviceOnce once;
    e = once.run([] { return cudaFuncSetAttribute(beam_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 << 10); });
    if (e != cudaSuccess) return e;
    e = launch_next(beam_join_kernel, dim3((uint32_t)job.batch), dim3(JOIN_THREADS + 32), room, stream, p);
    if (e == cudaSuccess) ++*launches;
    timing_mark(stream);
    return e;
}

cudaError_t launch_beam_reorder(const BeamReorderJob &job, cudaStream_t stream, int *launches) {
    // units as wide as every segment's start allows; its end may be shorter
    size_t all = reinterpret_cast<uintptr_t>(job.in) | reinterpret_cast<uintptr_t>(job.out);
    for (const size_t s : {job.in_outer, job.in_batch, job.in_beam, job.in_segment, job.out_outer, job.out_batch, job.out_beam, job.out_segment})
        all |= s;
    size_t word = 16;
    while (all % word != 0 || word > job.segment_bytes) word /= 2;
    ReorderParams p = {};
    p.rest = (uint32_t)(job.segment_bytes % word);
    p.parents = job.parents;
    p.beams = job.beams;
    p.into = job.into;
    p.in_outer = job.in_outer;
    p.in_batch = job.in_batch;
    p.in_beam = job.in_beam;
    p.in_segment = job.in_segment;
    p.out_outer = job.out_outer;
    p.out_batch = job.out_batch;
    p.out_beam = job.out_beam;
    p.out_segment = job.out_segment;
    p.place = job.in == job.out;
    const size_t units = (job.segment_bytes + word - 1) / word, each = job.batch * job.segments * units;
    p.unit = Divisor((uint32_t)units);
    p.segment = Divisor((uint32_t)job.segments);
    p.batch = Divisor((uint32_t)job.batch);
    // so many of the outer ones at a time that their places are counted in 32 bits
    const size_t most = ((size_t)1 << 31) / each > 0 ? ((size_t)1 << 31) / each : 1;
    for (size_t o = 0; o < job.outer; o += most) {
        const size_t count = job.outer - o < most ? job.outer - o : most;
        p.in = job.in + o * job.in_outer;
        p.out = job.out + o * job.out_outer;
        p.total = (uint32_t)(count * each);
        const cudaError_t e = word == 16  ? launch_reorder_by<uint4>(p, stream)
                              : word == 8 ? launch_reorder_by<uint64_t>(p, stream)
                              : word == 4 ? launch_reorder_by<uint32_t>(p, stream)
                              : word == 2 ? launch_reorder_by<uint16_t>(p, stream)
                                          : launch_reorder_by<uint8_t>(p, stream);
        if (e != cudaSuccess) return e;
        ++*launches;
        timing_mark(stream);
    }
    return cudaSuccess;
}

}  // namespace gbs
