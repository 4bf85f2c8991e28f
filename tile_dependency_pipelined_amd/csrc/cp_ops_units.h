// cp_ops_units.h -- 16-byte units of elements: stored in part, unpacked, packed; and the
// order of a wave's accesses to LDS.  Internal to the library.
#pragma once
#include "cp_ops_device.h"

namespace cpo {

// Between a wave's accesses to LDS by which its lanes pass values to each other.  They
// execute in order; the compiler, to which a lane's own stores are all there is, must
// keep it.  No instruction comes of it.
__device__ __forceinline__ void settle_lds() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The first `n` elements of a unit (all, if it has no more) to memory of any alignment.
template <class T>
__device__ __forceinline__ void store_partial(char *p, uint4 u, int n) {
    if (n >= kUnit<T>) {
        __builtin_memcpy(p, &u, 16);
    } else {
        T e[kUnit<T>];
        __builtin_memcpy(e, &u, 16);
#pragma unroll
        for (int i = 0; i < kUnit<T> - 1; ++i)
            if (i < n) reinterpret_cast<T *>(p)[i] = e[i];
    }
}
template <class T>
__device__ __forceinline__ void unpack_unit(uint4 u, float (&v)[kUnit<T>]) {
    T e[kUnit<T>];
    __builtin_memcpy(e, &u, 16);
#pragma unroll
    for (int i = 0; i < kUnit<T>; ++i) v[i] = to_f32(e[i]);
}
template <class T>
__device__ __forceinline__ uint4 pack_unit(const float (&v)[kUnit<T>]) {
    T e[kUnit<T>];
#pragma unroll
    for (int i = 0; i < kUnit<T>; ++i) e[i] = from_f32<T>(v[i]);
    uint4 u;
    __builtin_memcpy(&u, e, 16);
    return u;
}

}  // namespace cpo
