// common.cuh -- stands in for the kernels' own where they run on the host: a block's threads are host threads, one block
// after the other, on host memory.  What the cache's kernels use of CUDA, and no more.  Collectives take whole warps.
#pragma once

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <thread>
#include <vector>

#include <pthread.h>

#include <cuda_runtime_api.h>
#include <vector_functions.h>

#include "spec_reject.h"

#undef __device__
#undef __global__
#undef __shared__
#undef __host__
#undef __forceinline__
#undef __noinline__
#undef __launch_bounds__
#define __device__
#define __global__
#define __host__
#define __shared__ static
#define __forceinline__ inline
#define __noinline__
#define __launch_bounds__(...)

inline thread_local uint3 threadIdx, blockIdx;
inline dim3 blockDim, gridDim;

namespace emulated {

struct Barrier {
    pthread_barrier_t b;
    explicit Barrier(unsigned n) { pthread_barrier_init(&b, nullptr, n); }
    ~Barrier() { pthread_barrier_destroy(&b); }
    void wait() { pthread_barrier_wait(&b); }
};

struct Warp {
    Barrier all{32};
    int64_t value[32];
};

struct Block {
    Barrier all;
    std::vector<int> value;
    std::vector<Warp> warps;
    explicit Block(unsigned n) : all(n), value(n), warps((n + 31) / 32) {}
};

inline thread_local Block *here;

// Every lane's value, as lane `lane` sees it when all have come.
template <class F> auto with_warp(int64_t mine, F f)
{
    Warp &w = here->warps[threadIdx.x / 32];
    w.value[threadIdx.x % 32] = mine;
    w.all.wait();
    const auto y = f(w.value, (int)(threadIdx.x % 32));
    w.all.wait();
    return y;
}

template <class... P, class... A> cudaError_t launch(const cudaLaunchConfig_t *cfg, void (*kernel)(P...), A... args)
{
    gridDim = cfg->gridDim;
    blockDim = cfg->blockDim;
    for (unsigned y = 0; y < gridDim.y; ++y)
        for (unsigned x = 0; x < gridDim.x; ++x) {
            Block b(blockDim.x);
            std::vector<std::thread> threads;
            for (unsigned t = 0; t < blockDim.x; ++t)
                threads.emplace_back([&, t] {
                    threadIdx = uint3{t, 0, 0};
                    blockIdx = uint3{x, y, 0};
                    here = &b;
                    kernel(static_cast<P>(args)...);
                });
            for (auto &t : threads)
                t.join();
        }
    return cudaSuccess;
}

inline cudaError_t device(int *d) { return *d = 0, cudaSuccess; }
inline cudaError_t attribute(int *n, cudaDeviceAttr, int) { return *n = 2, cudaSuccess; }
inline cudaError_t none() { return cudaSuccess; }
inline cudaError_t copy(void *to, const void *from, size_t n, cudaMemcpyKind, cudaStream_t)
{
    return std::memcpy(to, from, n), cudaSuccess;
}
inline cudaError_t set(void *to, int x, size_t n, cudaStream_t) { return std::memset(to, x, n), cudaSuccess; }
inline cudaError_t wait(cudaStream_t) { return cudaSuccess; }

}  // namespace emulated

#define cudaLaunchKernelEx emulated::launch
#define cudaGetDevice emulated::device
#define cudaDeviceGetAttribute emulated::attribute
#define cudaPeekAtLastError emulated::none
#define cudaGetLastError emulated::none
#define cudaMemcpyAsync emulated::copy
#define cudaMemsetAsync emulated::set
#define cudaStreamSynchronize emulated::wait

using std::max;
using std::min;

inline void __syncthreads() { emulated::here->all.wait(); }
inline int __syncthreads_or(int x)
{
    auto &b = *emulated::here;
    b.value[threadIdx.x] = x;
    b.all.wait();
    const int y = std::any_of(b.value.begin(), b.value.end(), [](int v) { return v != 0; });
    b.all.wait();
    return y;
}
inline void __syncwarp() { emulated::here->warps[threadIdx.x / 32].all.wait(); }
inline void __threadfence() { std::atomic_thread_fence(std::memory_order_seq_cst); }
template <class T> T __shfl_sync(unsigned, T x, int from)
{
    return (T)emulated::with_warp((int64_t)x, [&](const int64_t *v, int) { return v[from & 31]; });
}
template <class T> T __shfl_up_sync(unsigned, T x, int d)
{
    return (T)emulated::with_warp((int64_t)x, [&](const int64_t *v, int lane) { return v[lane >= d ? lane - d : lane]; });
}
inline unsigned __ballot_sync(unsigned, int x)
{
    return emulated::with_warp(x != 0, [](const int64_t *v, int) {
        unsigned y = 0;
        for (int i = 0; i < 32; ++i)
            y |= (unsigned)v[i] << i;
        return y;
    });
}
inline int __any_sync(unsigned m, int x) { return __ballot_sync(m, x) != 0; }
inline int __all_sync(unsigned m, int x) { return __ballot_sync(m, x) == 0xffffffffu; }
inline int __popc(unsigned x) { return __builtin_popcount(x); }
inline int __ffs(int x) { return __builtin_ffs(x); }
inline int __clz(int x) { return x ? __builtin_clz((unsigned)x) : 32; }
template <class T> T __ldcg(const T *p) { return *p; }
template <class T> T atomicAdd(T *p, T x) { return __atomic_fetch_add(p, x, __ATOMIC_SEQ_CST); }
template <class T> T atomicSub(T *p, T x) { return __atomic_fetch_sub(p, x, __ATOMIC_SEQ_CST); }
template <class T, class U> T atomicOr(T *p, U x) { return __atomic_fetch_or(p, (T)x, __ATOMIC_SEQ_CST); }
template <class T> T atomicMin(T *p, T x)
{
    T old = __atomic_load_n(p, __ATOMIC_SEQ_CST);
    while (x < old && !__atomic_compare_exchange_n(p, &old, x, false, __ATOMIC_SEQ_CST, __ATOMIC_SEQ_CST)) {
    }
    return old;
}

namespace specrej {

constexpr unsigned kFull = 0xffffffffu;
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline uint4 ld_stream(const void *p) { return *static_cast<const uint4 *>(p); }

}  // namespace specrej
