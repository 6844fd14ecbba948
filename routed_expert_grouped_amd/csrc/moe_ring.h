// moe_ring.h -- helpers of the streaming kernels that keep a ring of register stages in flight.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace moe {

// A kernel argument as a global-memory pointer held in registers, and a choice between two of them by
// value: left to itself, a choice between two arguments becomes a load from the chosen argument's address,
// and waiting for that load would wait for the ring.
typedef const __attribute__((address_space(1))) uint8_t* gbytes;
template <typename V>
using gvec = const __attribute__((address_space(1))) V*;

__device__ __forceinline__ gbytes held(const void* p) {
    uint64_t v = (uint64_t)p;
    asm("" : "+s"(v));
    return (gbytes)v;
}
template <typename P>
__device__ __forceinline__ P pick(bool c, P a, P b) {
    return c ? a : b;
}

// f of slots 0 .. D - 1
template <int D, int d = 0, typename F>
__device__ __forceinline__ void each_slot(F&& f) {
    f(std::integral_constant<int, d>{});
    if constexpr (d + 1 < D) each_slot<D, d + 1>(f);
}

// n stages through a ring of D slots.  The loop goes round whole and has one exit, so that the compiler
// sees every slot's loads behind the others' and its waits leave those in flight; the last n % D
// stages follow it.
template <int D, typename F>
__device__ __forceinline__ void ring_loop(int n, F&& slot) {
    int i = 0;
    for (; i + D <= n; i += D) each_slot<D>(slot);
    each_slot<D - 1>([&](auto tag) {
        if (i + decltype(tag)::value < n) slot(tag);
    });
}

}  // namespace moe
