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
        asm("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t@q ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
            : "+r"(w[0]), "+r"(w[1]), "+r"(w[2]), "+r"(w[3])
            : "l"(p), "r"((uint32_t)on));
    } else if constexpr (BYTES == 8) {
        asm("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %3, 0;\n\t@q ld.global.nc.v2.u32 {%0, %1}, [%2];\n\t}"
            : "+r"(w[0]), "+r"(w[1])
            : "l"(p), "r"((uint32_t)on));
    } else if constexpr (BYTES == 4) {
        asm("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q ld.global.nc.u32 %0, [%1];\n\t}"
            : "+r"(w[0])
            : "l"(p), "r"((uint32_t)on));
    } else {
        if (on) x = load_pack<T, N>(p);
    }
    return x;
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
// value overflows: an id below `first` wraps to a value above any count.
__device__ __forceinline__ int32_t id_index(const void *ids, int id_bytes, size_t i, int64_t first, uint64_t count) {
    const int64_t id = id_bytes == 8 ? static_cast<const int64_t *>(ids)[i] : static_cast<const int32_t *>(ids)[i];
    const uint64_t at = (uint64_t)id - (uint64_t)first;
    return at < count ? (int32_t)at : -1;
}

template <typename ID> __device__ __forceinline__ int32_t id_index(const ID *ids, size_t i, int64_t first, uint64_t count) {
    const uint64_t at = (uint64_t)(int64_t)ids[i] - (uint64_t)first;
    return at < count ? (int32_t)at : -1;
}

// The table row of an id as a key: `vocab` for ids that have none.
template <typename ID> __device__ __forceinline__ uint32_t id_key(const ID *ids, size_t i, int64_t first, int64_t padding, uint32_t vocab) {
    const int64_t id = ids[i];
    const uint64_t at = (uint64_t)id - (uint64_t)first;
    return at < vocab && !(padding >= 0 && id == padding) ? (uint32_t)at : vocab;
}

// A kernel of a call's later steps is launched while the one before it still
// runs (launch_next below): it waits here, before it reads or writes anything
// that an earlier kernel does, and lets the kernel after it be launched.
__device__ __forceinline__ void wait_for_earlier() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A router weight in 32 bits; 1 without weights.
template <typename W> __device__ __forceinline__ float weight_at(const W *w, size_t i) {
    return w ? to_f32(w[i]) : 1.0f;
}

// Launches a step that begins with wait_for_earlier(), after another step of
// the same call on the same stream.
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
