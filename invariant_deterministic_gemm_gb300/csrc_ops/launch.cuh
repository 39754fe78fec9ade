// Launches that begin while the one in front of them ends.
//
// Every kernel here waits at its top for the launch in front to be over, before
// it touches memory, and one of few blocks lets the next launch of its stream
// begin as soon as all its own blocks are running. What a launch costs besides
// its work (about 2 us: its set-up, its blocks' way to the SMs) then overlaps
// the work in front: an embedding of 333 tokens with its gradient, four
// launches, takes 30.6 us and took 39.5. A launch that waits is over after the
// one it waited for, so a chain of them keeps the stream's order; behind a
// kernel that lets nothing begin early, or in front of one that is launched
// without the attribute, the order is the ordinary one.
//
// Inputs are read with plain loads, never through the read-only path (__ldg):
// that takes for granted that nothing is written from a launch's begin on, and
// these begin before their inputs are complete.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace deto {

__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Letting the next begin costs a large grid more than it saves: a lookup of
// 8192 rows (32768 blocks) 34 us instead of 20. The 8-bit products have rules of
// their own: the tile of few rows lets the next begin when its last copies are
// under way (quantiser and product of three rows 14.7 instead of 16.4 us; at its
// start the next blocks take the room of its own, 12.2 instead of 10.3 us for
// the product), the plain tile never (ragged prefill 60.1 us without, 62.1 with).
constexpr unsigned kFewBlocks = 2048;
__device__ __forceinline__ void begin()
{
    if (gridDim.x <= kFewBlocks) let_next_begin();
    wait_for_last();
}

// Runs `set_up` once per device for one kernel instance (its state in `done`).
template <typename F>
cudaError_t once_per_device(std::atomic<uint64_t> &done, F set_up)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = set_up();
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// cluster: CTAs of a cluster (1: none).
template <typename... P, typename... A>
cudaError_t launch_early(void (*fn)(P...), long long grid, int threads, size_t smem, int cluster, cudaStream_t s, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, args...);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace deto
