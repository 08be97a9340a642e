// Rows of 32- and 16-bit floating point values: conversions, vectors of a
// row's values and the choice of their width.  Shared by the kernels that
// move and sum rows in sorted order (expert.cu, embedding.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "rows.h"

namespace gbs {
namespace {

// Values of a row type in 32 bits and back (one rounding, to nearest even).
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// N consecutive values, loaded and stored as one access (two for 32 bytes).
template <typename T, int N> struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Pack {
    T v[N];
};
template <typename T, int N> __device__ __forceinline__ Pack<T, N> load_pack(const T *p) {
    return *reinterpret_cast<const Pack<T, N> *>(p);
}
template <typename T, int N> __device__ __forceinline__ void store_pack(T *p, const Pack<T, N> &x) {
    *reinterpret_cast<Pack<T, N> *>(p) = x;
}

// The pack at p where `on`, zeros elsewhere, as one predicated access: a row's
// loads then leave together, with no branch between them.
template <typename T, int N> __device__ __forceinline__ Pack<T, N> load_pack_if(const T *p, bool on) {
    Pack<T, N> x = Pack<T, N>{};
    constexpr int BYTES = N * (int)sizeof(T);
    uint32_t *w = reinterpret_cast<uint32_t *>(&x);
    if constexpr (BYTES == 16) {
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t@q ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
            : "+r"(w[0]), "+r"(w[1]), "+r"(w[2]), "+r"(w[3])
            : "l"(p), "r"((uint32_t)on));
    } else if constexpr (BYTES == 8) {
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %3, 0;\n\t@q ld.global.v2.u32 {%0, %1}, [%2];\n\t}"
            : "+r"(w[0]), "+r"(w[1])
            : "l"(p), "r"((uint32_t)on));
    } else if constexpr (BYTES == 4) {
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q ld.global.u32 %0, [%1];\n\t}"
            : "+r"(w[0])
            : "l"(p), "r"((uint32_t)on));
    } else {
        if (on) x = load_pack<T, N>(p);
    }
    return x;
}

// ---------------------------------------------------------------------------
// Rows at any place
// ---------------------------------------------------------------------------
//
// Rows whose starts or lengths are not multiples of 16 bytes (ODD below) are
// still read and written 16 aligned bytes at a time: a pack is cut out of two
// neighbouring words, and the packs of a row's part go through shared memory,
// from where they are written as aligned words, the part's ends two bytes at a
// time.  An aligned word that holds a byte of the row lies in the allocation's
// granule, whatever else it holds; only the row's own bytes are used, and only
// they are written.

// The 16 bytes from byte a (even, below 16) of the 32 bytes in w, in w[0..3].
__device__ __forceinline__ void shift_bytes(uint32_t (&w)[8], uint32_t a) {
    if (a & 8)
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    if (a & 4)
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    if (a & 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
}

// The pack of 16 bytes at p, of which `left` values (any more than a pack
// count as one) are the row's; zeros elsewhere.
template <typename T> __device__ __forceinline__ Pack<T, 16 / sizeof(T)> load_odd(const T *p, int32_t left, bool on) {
    constexpr int N = 16 / (int)sizeof(T);
    using Q = Pack<uint32_t, 4>;
    const uint32_t a = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15;
    const uint32_t *q = reinterpret_cast<const uint32_t *>(reinterpret_cast<uintptr_t>(p) - a);
    on = on && left > 0;
    const int32_t mine = left < N ? left : N;
    const Q x = load_pack_if<uint32_t, 4>(q, on), y = load_pack_if<uint32_t, 4>(q + 4, on && (int32_t)a + mine * (int32_t)sizeof(T) > 16);
    uint32_t w[8] = {x.v[0], x.v[1], x.v[2], x.v[3], y.v[0], y.v[1], y.v[2], y.v[3]};
    shift_bytes(w, a);
    Pack<T, N> r;
    *reinterpret_cast<uint4 *>(&r) = make_uint4(w[0], w[1], w[2], w[3]);
    if (left < N)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i >= left) r.v[i] = T{};
    return r;
}

// A pack of a row of row_len values from column c on.
template <bool ODD, typename T> __device__ __forceinline__ Pack<T, 16 / sizeof(T)> load_row(const T *row, uint32_t c, uint32_t row_len, bool on) {
    if constexpr (ODD) return load_odd<T>(row + c, (int32_t)row_len - (int32_t)c, on);
    else return load_pack_if<T, 16 / (int)sizeof(T)>(row + c, on && c < row_len);
}

// Writes `bytes` (even) bytes of a row's part to dst (even): those from byte
// `from` on of shared memory at st (16-byte aligned, readable for 31 bytes
// after them).  `lanes` lanes take part, this one as `sub`.
__device__ __forceinline__ void write_part(unsigned char *dst, const unsigned char *st, uint32_t from, uint32_t bytes, uint32_t sub, uint32_t lanes) {
    const uint32_t b = (uint32_t)reinterpret_cast<uintptr_t>(dst) & 15, head = min(b ? 16 - b : 0, bytes);
    for (uint32_t i = 2 * sub; i < head; i += 2 * lanes) *reinterpret_cast<uint16_t *>(dst + i) = *reinterpret_cast<const uint16_t *>(st + from + i);
    const uint32_t a = (from + head) & 15, first = from + head - a, whole = (bytes - head) & ~15u;
    for (uint32_t i = 16 * sub; i < whole; i += 16 * lanes) {
        const uint4 x = *reinterpret_cast<const uint4 *>(st + first + i), y = *reinterpret_cast<const uint4 *>(st + first + i + 16);
        uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        shift_bytes(w, a);
        *reinterpret_cast<uint4 *>(dst + head + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    for (uint32_t i = head + whole + 2 * sub; i < bytes; i += 2 * lanes)
        *reinterpret_cast<uint16_t *>(dst + i) = *reinterpret_cast<const uint16_t *>(st + from + i);
}
constexpr uint32_t PART_PAD = 32;  // bytes after a part in shared memory
// Fewest lanes that share a row at any place: few parts in a warp's shared memory.
constexpr uint32_t ODD_LOG_LANES = 3;

// A pack of a row's part on its way out: to the row, or (ODD) to its place in shared memory.
template <bool ODD, typename T, int N>
__device__ __forceinline__ void put_pack(T *row, uint32_t c, uint32_t row_len, const Pack<T, N> &x, bool on, unsigned char *st, uint32_t index) {
    if constexpr (ODD) *reinterpret_cast<uint4 *>(st + 16 * index) = *reinterpret_cast<const uint4 *>(&x);
    else if (on && c < row_len) store_pack(row + c, x);
}
// The bytes of a row's part of `most` values from column c on.
template <typename T> __device__ __forceinline__ uint32_t part_bytes(uint32_t c, uint32_t most, uint32_t row_len) {
    return (c >= row_len ? 0 : min(most, row_len - c)) * (uint32_t)sizeof(T);
}

// Zeroes `bytes` (even) from p on, 16 aligned bytes at a time; a warp's work.
__device__ __forceinline__ void zero_bytes(unsigned char *p, size_t bytes) {
    const uint32_t lane = threadIdx.x & 31;
    const size_t a = reinterpret_cast<uintptr_t>(p) & 15, head = a ? (16 - a < bytes ? 16 - a : bytes) : 0, whole = (bytes - head) / 16 * 16;
    for (size_t i = 16 * lane; i < whole; i += 512) *reinterpret_cast<uint4 *>(p + head + i) = make_uint4(0, 0, 0, 0);
    if (2 * lane < head) *reinterpret_cast<uint16_t *>(p + 2 * lane) = 0;
    if (2 * lane < bytes - head - whole) *reinterpret_cast<uint16_t *>(p + head + whole + 2 * lane) = 0;
}

// The same for memory that this kernel writes too, packs of 16 or 32 bytes or less than 16.
template <typename T, int N> __device__ __forceinline__ Pack<T, N> load_own_if(const T *p, bool on) {
    Pack<T, N> x = Pack<T, N>{};
    constexpr int BYTES = N * (int)sizeof(T);
    uint32_t *w = reinterpret_cast<uint32_t *>(&x);
    if constexpr (BYTES >= 16) {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i)
            asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t@q ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                         : "+r"(w[4 * i]), "+r"(w[4 * i + 1]), "+r"(w[4 * i + 2]), "+r"(w[4 * i + 3])
                         : "l"(reinterpret_cast<const char *>(p) + 16 * i), "r"((uint32_t)on)
                         : "memory");
    } else {
        if (on) x = load_pack<T, N>(p);
    }
    return x;
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A slot's id as an index into [0, count), or -1 where it lies outside.  The
// subtraction is done in 64 bits without sign, so that no id and no first
// value overflows: an id below `first` wraps to a value above any count that
// ids_from (rows.h) gives.
__device__ __forceinline__ int32_t id_index(const void *ids, int id_bytes, size_t i, int64_t first, uint64_t count) {
    const int64_t id = id_bytes == 8 ? static_cast<const int64_t *>(ids)[i] : static_cast<const int32_t *>(ids)[i];
    const uint64_t at = (uint64_t)id - (uint64_t)first;
    return at < count ? (int32_t)at : -1;
}

template <typename ID> __device__ __forceinline__ int32_t id_index(const ID *ids, size_t i, int64_t first, uint64_t count) {
    const uint64_t at = (uint64_t)(int64_t)ids[i] - (uint64_t)first;
    return at < count ? (int32_t)at : -1;
}

// The table row of an id as a key, one of the first `inside`: `vocab` for ids that have none.
__device__ __forceinline__ uint32_t id_key(int64_t id, int64_t first, int64_t padding, uint32_t inside, uint32_t vocab) {
    const uint64_t at = (uint64_t)id - (uint64_t)first;
    return at < inside && (padding < 0 || id != padding) ? (uint32_t)at : vocab;
}
// The keys of a whole list into shared memory, ~0 from n to `most`; a CTA's
// work.  The ids of a thread's turn are fetched together.
template <typename ID>
__device__ __forceinline__ void load_keys(uint32_t *key, const ID *ids, uint32_t n, uint32_t most, int64_t first, int64_t padding, uint32_t inside,
                                          uint32_t vocab) {
    constexpr int U = 8;
    for (uint32_t i0 = threadIdx.x; i0 < most; i0 += U * blockDim.x) {
        ID id[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t i = i0 + j * blockDim.x;
            id[j] = ids[i < n ? i : 0];
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t i = i0 + j * blockDim.x;
            if (i < most) key[i] = i < n ? id_key(id[j], first, padding, inside, vocab) : ~0u;
        }
    }
}

// A kernel may be launched while the one before it on the stream still ends
// (launch_next below): all of its threads that touch global memory wait here
// first, for all that earlier kernels do.  What a call's rows come from can be
// written by the kernel before, so their loads keep behind the wait (volatile)
// and out of the read-only path.  Calls in a row, us a call: a gradient of 999
// ids 7.3, launched plainly 10.2; of 8192 ids 53.8 and 61.7; combine's gradient of
// 2047 f32 tokens 8.1 and 10.3.
__device__ __forceinline__ void wait_for_earlier() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel's CTAs take their places now rather than as this one
// ends.  Only the steps of an order do (8192 ids 53.8 us, without 54.0): behind a
// kernel that moves rows the early CTAs crowd on the SMs that finish first
// (a gradient of 999 ids 9.9 us instead of 7.3, dispatch of 4095 tokens 24.8
// instead of 24.3).
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A router weight in 32 bits; 1 without weights.
template <typename W> __device__ __forceinline__ float weight_at(const W *w, size_t i) {
    return w ? to_f32(w[i]) : 1.0f;
}

// Launches a kernel that begins with wait_for_earlier().  Behind a kernel that
// does not let the next one be launched (another library's) it begins as that
// one ends.
template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace
}  // namespace gbs
