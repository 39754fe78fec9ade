// Launches that begin while the one in front of them ends.
//
// Every kernel here waits at its top for the launch in front to be over, before
// it touches memory, and one of few blocks lets the next launch of its stream
// begin as soon as all its own blocks are running. What a launch costs besides
// its work (its set-up, its blocks' way to the SMs) then overlaps the work in
// front: an embedding of 333 tokens with its gradient, four launches, takes 27.6
// us and 37.4 without; routing, dispatch, gather and combine of 17 tokens out of a
// graph 9.0 and 9.8. A launch that waits is over after the one it waited for, so
// a chain of them keeps the stream's order; behind a kernel that lets nothing
// begin early, or in front of one that is launched without the attribute, the
// order is the ordinary one.
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

// Few blocks are fewer than there are SMs: the waiting blocks of the next launch
// then have SMs to themselves. Quantiser and product of 64 rows (64 blocks, then
// the product's) 12.3 us out of a graph, 13.5 if nothing lets the next begin; the
// layer above of 256 tokens (gather 128 blocks, combine 256) 9.1, and 10.0 if up to
// 2048 blocks do. A larger grid's own blocks make room for blocks that wait: a
// lookup of 256 rows (1024 blocks) 2.25 us either way, 512 rows 2.4 without and 3.2
// with, 1024 rows 3.5 and 5.2, 8192 rows 25 and 34; the prompt's quantiser and product
// 57.2 and 58.4. The 8-bit products have rules of their own: the tile of few rows
// lets the next begin when its last copies are under way (quantiser and product of
// three rows 14.7 instead of 16.4 us; at its start the next blocks take the room
// of its own, 12.2 instead of 10.3 us for the product), the plain tile never
// (ragged prefill 60.1 us without, 62.1 with).
constexpr unsigned kFewBlocks = 128;
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
