// Access to LDS by address, copies into it that bypass the registers, and waits.
#pragma once

#include "w4a16_device.hpp"

namespace w4a16 {
namespace {

typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) void lds_void;
template <typename T>
__device__ __forceinline__ T lds_get(const lds_u8 *p) {
    return *reinterpret_cast<const __attribute__((address_space(3))) T *>(p);
}
template <typename T>
__device__ __forceinline__ void lds_put(lds_u8 *p, T v) {
    *reinterpret_cast<__attribute__((address_space(3))) T *>(p) = v;
}

// One KiB from `base + at` to LDS without passing through registers, lane l's 16 bytes to 16 l; what
// lies at or past base + bytes comes as zeros.
__device__ __forceinline__ void copy_kib(const uint8_t *base, uint32_t bytes, uint32_t at, lds_u8 *to, int lane) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(base, bytes), (lds_void *)to, 16, 16 * lane, at, 0, 0);
}

// A workgroup barrier for LDS alone: this wave's LDS operations are done, and loads from memory
// stay under way (__syncthreads waits for those too).
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// s_waitcnt vmcnt(n): at most n of this wave's vector memory instructions are still under way.
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N < 64, "six bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

}  // namespace
}  // namespace w4a16
