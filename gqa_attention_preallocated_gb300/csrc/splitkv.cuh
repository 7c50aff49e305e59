// What the split-KV kernels share: the call's work partition as a kernel sees
// it, the walk over a CTA's tiles, and the chained launch.
#pragma once

#include <cuda_runtime.h>

#include <utility>

#include "kvc_internal.h"

namespace kvc {

// The call's work partition, read only after the grid-dependency wait.
// Part<false>: planned on the host, in the kernel parameters (indexed in
// parameter space).  Part<true>: planned on the device from device-resident
// lengths (a DevicePlan in the workspace).
template <bool DP>
struct Part;

template <>
struct Part<false> {
    const DecodeParams& p;
    __device__ __forceinline__ int gstart(int i) const { return p.gstart[i]; }
    __device__ __forceinline__ int prior(int b) const { return p.prior[b]; }
    __device__ __forceinline__ int n_new(int b) const { return p.n_new[b]; }
    __device__ __forceinline__ int total_tiles() const { return p.total_tiles; }
    __device__ __forceinline__ int NB() const { return p.NB; }
    __device__ __forceinline__ int Hkv() const { return p.Hkv; }
};

template <>
struct Part<true> {
    const DecodeParams& p;
    __device__ __forceinline__ int gstart(int i) const { return p.dplan->gstart[i]; }
    __device__ __forceinline__ int prior(int b) const { return p.dplan->prior[b]; }
    __device__ __forceinline__ int n_new(int b) const { return p.dplan->n_new[b]; }
    __device__ __forceinline__ int total_tiles() const { return p.dplan->total_tiles; }
    __device__ __forceinline__ int NB() const { return p.NB; }
    __device__ __forceinline__ int Hkv() const { return p.Hkv; }
};

// First key tile (absolute position / 64) of group q's units: 0, or with a
// window the tile holding the window start of the block's earliest query
// (the same rule as the planners'; tiles before it are never scheduled).
template <bool DP, int KT>
__device__ __forceinline__ int first_tile(const Part<DP>& w, int q) {
    const DecodeParams& p = w.p;
    if (p.window <= 0) return 0;
    const int b = q / p.RB, rb = q - b * p.RB;
    const int prior = w.prior(b), nn = w.n_new(b);
    const int r0 = rb * p.RPB, r1 = min(p.R, r0 + p.RPB);
    int qmin = 0x7fffffff;
    if (r1 - r0 >= p.T) {
        if (nn > 0) qmin = prior;
    } else {
        for (int r = r0; r < r1; ++r)
            if (r % p.T < nn) qmin = min(qmin, prior + r % p.T);
    }
    return qmin == 0x7fffffff ? 0 : max(0, qmin - p.window + 1) / KT;
}

// Largest q with gstart[q] <= x (gstart nondecreasing, x < gstart[NB]).
template <bool DP>
__device__ __forceinline__ int locate_group(const Part<DP>& w, int x) {
    int lo = 0, hi = w.NB();
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (w.gstart(mid) <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

template <bool DP, int KT>
struct Cursor {
    int q, kvh, j, nt, t0;  // t0: the group's first key tile
    __device__ __forceinline__ void init(const Part<DP>& w, int x) {
        q = locate_group(w, x);
        nt = (w.gstart(q + 1) - w.gstart(q)) / w.Hkv();
        const int off = x - w.gstart(q);
        kvh = off / nt;
        j = off - kvh * nt;
        t0 = first_tile<DP, KT>(w, q);
    }
    __device__ __forceinline__ void advance(const Part<DP>& w) {
        if (++j < nt) return;
        j = 0;
        if (++kvh < w.Hkv()) return;
        kvh = 0;
        ++q;
        while (q < w.NB() && w.gstart(q + 1) == w.gstart(q)) ++q;
        if (q < w.NB()) {
            nt = (w.gstart(q + 1) - w.gstart(q)) / w.Hkv();
            t0 = first_tile<DP, KT>(w, q);
        }
    }
};

// Row (of the cache's 2-D view) of the key at absolute position a of unit
// (b, kvh): contiguous, ring (a mod max_len) or paged (through the block
// table).  Tiles never straddle a ring wrap or a page (max_len / page are
// multiples of the tile size there).  A bad table entry records an error.
__device__ __forceinline__ int key_row(const DecodeParams& p, int b, int kvh, int a) {
    bool bad = false;
    const int row = phys_row(p.pg, p.ring, p.Hkv, p.max_len, b, kvh, a, &bad);
    if (bad) atomicExch(p.err, kDevBadPage);
    return row;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
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
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace kvc
