// Splitting one tile's work over the blocks of a cluster.
//
// O, dQ, dK and dV of a tile are plain sums over the tiles it streams (sigma has no
// normalisation to carry along), so a batch with too few tiles to fill the device
// gives each of them to a cluster: block r takes the r-th part of the steps, leaves
// its fp32 sums in shared memory, and after a cluster barrier every block adds
// up its share of the columns over distributed shared memory, in the order of the
// blocks, and rounds once.  Nothing passes through global memory, and the result
// does not depend on scheduling.  The split kernels are instances of their own:
// as a run-time choice the code cost the other batches 2 to 7% at D = 64.
#pragma once

#include "sm100.cuh"

namespace sigattn {

// Clusters of eight blocks were slower than of four in every shape tried (32 tiles of
// 1024 to 4096 keys at D = 128, forward: 29.6 us in fours, 52.2 in eights): few of them
// fit the device at a time.
constexpr unsigned kMostSplit = 4;

// Block of the cluster, and its place in a grid whose x axis is `split` times as wide.
struct SplitPlace {
    int rank, x, wide;    // rank in the cluster; blockIdx.x and gridDim.x without the split
};
__device__ __forceinline__ SplitPlace split_place(int split) {
    SplitPlace s{0, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x)};
    if (split > 1) {
        s.rank = s.x % split;
        s.x /= split;
        s.wide /= split;
    }
    return s;
}
// First step of block `rank` of `split`, of `steps`.
__device__ __forceinline__ int split_step(int steps, int rank, int split) {
    return static_cast<int>(static_cast<int64_t>(steps) * rank / split);
}

// Barrier over all threads of the cluster's blocks, with their shared memory.  The
// .aligned form wants whole warps, and rows that end inside a warp's may have split
// the caller's.
__device__ __forceinline__ void cluster_meet() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// What a block does that has nothing to add or to leave: its shared memory has to
// outlive the others' reads, should they find rows that see keys (spans written by
// another stream meanwhile give wrong results, but must not fault).
__device__ __forceinline__ void cluster_skip() {
    cluster_meet();
    cluster_meet();
}
// 16 bytes at this block's shared address `a`, of block `rank`.
__device__ __forceinline__ float4 cluster_load(uint32_t a, int rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [r];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(a), "r"(rank)
        : "memory");
    return v;
}

// Partial sums in shared memory: [column / 4][128 rows] float4, so that the lanes
// of a warp, which hold a row each, write side by side.  Leaves `cols` columns
// of this thread's row, from column `col` on, out of tensor memory (or zeros).
__device__ __forceinline__ void split_leave(float4 *sums, uint32_t taddr, int col, int cols, int row, bool zero) {
    for (int c = 0; c < cols; c += 32) {
        uint32_t r[32];
        if (!zero) tmem_ld32(taddr + c, r);
        float4 *to = sums + static_cast<size_t>((col + c) / 4) * 128 + row;
#pragma unroll
        for (int v = 0; v < 8; ++v)
            to[v * 128] = zero ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                               : make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                                             __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3]));
    }
}
// Adds up this block's share of `octets` groups of eight columns, thread `tid` of
// `threads`; f(group, row, sums) stores them.
template <typename F>
__device__ __forceinline__ void split_add(const float4 *sums, int octets, int rank, int split, int tid, int threads,
                                          F &&f) {
    const int first = octets * rank / split, last = octets * (rank + 1) / split;
    for (int e = first * 128 + tid; e < last * 128; e += threads) {
        const int octet = e / 128, row = e % 128;
        const uint32_t a = smem_u32(sums + static_cast<size_t>(2 * octet) * 128 + row);
        float x[8] = {};
        for (int r = 0; r < split; ++r) {
            const float4 lo = cluster_load(a, r), hi = cluster_load(a + 128 * sizeof(float4), r);
            x[0] += lo.x;
            x[1] += lo.y;
            x[2] += lo.z;
            x[3] += lo.w;
            x[4] += hi.x;
            x[5] += hi.y;
            x[6] += hi.z;
            x[7] += hi.w;
        }
        f(octet, row, x);
    }
}
__device__ __forceinline__ uint4 split_pack(const float (&x)[8], float scale, bool valid) {
    if (!valid) return make_uint4(0u, 0u, 0u, 0u);
    return make_uint4(pack_bf16x2(scale * x[0], scale * x[1]), pack_bf16x2(scale * x[2], scale * x[3]),
                      pack_bf16x2(scale * x[4], scale * x[5]), pack_bf16x2(scale * x[6], scale * x[7]));
}

}  // namespace sigattn
