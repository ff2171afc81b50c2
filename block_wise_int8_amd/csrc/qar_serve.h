// qar_serve.h -- what the serving kernels (qar_kv8.hip, qar_mx4.hip) share
// beside qar_device.h.
#pragma once

#include <hip/hip_runtime.h>

#include <tuple>
#include <type_traits>
#include <utility>

namespace qar {

constexpr int kDppRowRotate8 = 0x128;    // lane i <-> i ^ 8 within each 16 lanes

// Launches k<<<blocks, threads, 0, st>>>(a...) and returns that launch's
// own status, not an error that an unrelated call left on the thread.
template <typename... P, typename... A>
hipError_t launch_threads(void (*k)(P...), uint32_t blocks, uint32_t threads, hipStream_t st, A&&... a) {
    static_assert(sizeof...(P) == sizeof...(A), "kernel argument count");
    std::tuple<std::decay_t<P>...> vals(static_cast<std::decay_t<P>>(std::forward<A>(a))...);
    void* args[sizeof...(P)];
    std::apply([&](auto&... v) {
        size_t i = 0;
        ((args[i++] = static_cast<void*>(&v)), ...);
    }, vals);
    return hipLaunchKernel(reinterpret_cast<const void*>(k), dim3(blocks), dim3(threads), args, 0, st);
}

} // namespace qar
