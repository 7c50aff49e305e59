// What the split-KV kernels of 4-bit caches share: tile geometry, the loads and
// moves of packed codes, the producers, and the append of a chunk's rows.
#pragma once

#include <cuda_fp16.h>
#include <math.h>

#include "kvc_internal.h"
#include "ptx.cuh"
#include "q4.cuh"
#include "splitkv.cuh"

namespace kvc {
namespace q4 {

constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kLazyRescale = 8.0f;  // log2 of the largest factor p may reach above the reference
constexpr int kKT = kQ4KeyTile;       // keys per tile
constexpr int kWarpKeys = 32;
constexpr uint32_t kMinExp = 6;       // 2^(133 - 6) is the largest power of two of an fp32
constexpr int kTileWarps = kKT / kWarpKeys;  // warps that share a tile (a group)


// A stage of the ring: K's codes, V's codes, K's scale words, V's scale words.
template <int D>
struct Stage {
    static constexpr int kRowB = D / 2;         // bytes of a row's codes
    static constexpr int kCodeB = kKT * kRowB;  // one tile's K (or V) codes
    static constexpr int kBytes = 2 * kCodeB + 2 * kKT * 4;
};

// What a segment's end needs of its beginning (in shared memory).
struct Segment {
    unsigned long long row0;  // first query row of the block in q and out
    int flag[2];              // finish_unit's
    uint32_t valid;           // the block's rows that are queries
    int unit, unit_tile;      // the unit and its first tile
    int pad;
};
static_assert(sizeof(Segment) == 32, "shared memory map");

// Who works on a segment together.  Joint: the CTA's groups, tiles in turn.  Split
// (more parts than CTAs): every group has tiles of its own, and one group's
// segment ends while the others compute.  (Two kernels: with the choice made
// inside one, long decodes ran 7 % slower.)
template <int kGroups, bool split>
struct Party {
    int grp;
    __device__ __forceinline__ int part() const { return split ? grp * gridDim.x + blockIdx.x : blockIdx.x; }
    __device__ __forceinline__ int first_tile() const { return split ? 0 : grp; }
    static __device__ __forceinline__ constexpr int step() { return split ? 1 : kGroups; }
    static __device__ __forceinline__ constexpr int threads() { return split ? kTileWarps * 32 : kGroups * kTileWarps * 32; }
    __device__ __forceinline__ int rank(int tid) const { return split ? tid % (kTileWarps * 32) : tid; }
    __device__ __forceinline__ int lead() const { return split ? grp : 0; }  // the party's groups: lead() ..
    __device__ __forceinline__ int end() const { return split ? grp + 1 : kGroups; }
    __device__ __forceinline__ void sync() const { ptx::named_barrier_sync(split ? 2 + grp : 1, threads()); }
};

// Shares of the call's tiles.  (With the counters every share of a unit's range
// must have a tile: no more shares than tiles, as the host's plan has it.)
template <bool DP>
__device__ __forceinline__ int shares(const Part<DP>& w) {
    return DP && w.p.counters ? min(w.p.num_ctas, max(w.total_tiles(), 1)) : w.p.num_ctas;
}

// Key of row i (0 .. 7) of an 8-key block, a nibble each.
template <int D>
__device__ __forceinline__ int perm8(int i) {
    return ((D == 128 ? 0x67235410u : 0x67453210u) >> (4 * i)) & 7;
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}
// A scale word's zero point as a float.
__device__ __forceinline__ float zero_f32(uint32_t scale_word) {
    return __uint_as_float(0x4B000000u | (scale_word & 15u)) - 8388608.0f;
}
// Two keys' zero points as an f16 pair, z 2^-24 like the codes (an f16 subnormal).
__device__ __forceinline__ uint32_t zero_pair(uint32_t word_a, uint32_t word_b) {
    return ptx::prmt(word_a, word_b, 0x5410u) & 0x000F000Fu;
}

// What a row block's queries see: one past the last visible key, and the
// smallest last key of a valid query (no key, and a large one, without any).
template <bool DP>
__device__ __forceinline__ void block_bounds(const Part<DP>& w, int b, int rb, int& extent, int& min_lim) {
    const DecodeParams& p = w.p;
    const int prior = w.prior(b), nn = w.n_new(b);
    const int r0 = rb * p.RPB, n = min(p.R, r0 + p.RPB) - r0;  // rows r0 .. r0 + n - 1, query r % T each
    int t0 = 0, t1 = min(p.T, nn);  // the block's queries that exist lie in t0 .. t1 - 1, both ends among them
    if (n < p.T) {
        const int first = r0 % p.T, end = first + n;
        if (end <= p.T) {
            t0 = first;
            t1 = min(end, nn);
        } else if (nn <= first) {  // queries first .. T - 1 and 0 .. end - T - 1, of which the first part is padding
            t1 = min(end - p.T, nn);
        }
    }
    const bool any = t0 < t1;
    extent = any ? prior + t1 : 0;
    min_lim = any ? prior + t0 : 0x7fffffff;
}

// Padded queries (t >= n_new[b]) output zeros; spread over the whole grid.
template <int D, bool DP>
__device__ __forceinline__ void zero_padded_queries(const DecodeParams& p, const Part<DP>& wp, int tid, int threads) {
    const int rows_total = p.B * p.Hq * p.T;
    for (int row = blockIdx.x * threads + tid; row < rows_total; row += gridDim.x * threads) {
        const int t = row % p.T;
        const int b = row / (p.Hq * p.T);
        if (t >= wp.n_new(b)) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + static_cast<size_t>(row) * D);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

// Four dims of a query row's merged state: the output (row `row` of out, [B Hq T, d]),
// or this part's partial.
template <int D>
__device__ __forceinline__ void write_row(const DecodeParams& p, size_t row, int c4, float4 acc, float M, float L, bool sole,
                                          int slot, int lr) {
    if (sole) {
        const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // (NaN stays)
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + row * D + c4 * 4;
        uint2 v;
        v.x = ptx::pack_bf16x2(acc.x * inv, acc.y * inv);
        v.y = ptx::pack_bf16x2(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(dst) = v;
        return;
    }
    float* part = p.partials + (static_cast<size_t>(slot) * p.part_rows + lr) * (D + 4);
    reinterpret_cast<float4*>(part)[c4] = acc;
    if (c4 == 0) {
        part[D] = M;
        part[D + 1] = L;
    }
}

// The end of a unit of which this party saw a part: the last party to leave its
// partial merges all of them, in the order of the parts, and writes the unit's
// output.  Called by all the party's threads, after the partial's writes; `flag`
// is two ints of its shared memory.  unit = (group q, KV head kvh), us its
// first tile of N, ntiles its tiles; P parts.  p.counters returns to zero.
template <int D, int kRows, int kGroups, bool kSplit>
__device__ __forceinline__ void finish_unit(const DecodeParams& p, int unit, long long us, int ntiles, long long N, long long P,
                                            size_t row0, uint32_t valid, const Party<kGroups, kSplit>& party, int rank, volatile int* flag) {
    constexpr int PS = D + 4, C4 = D / 4, kChunk = 8;
    __threadfence();
    party.sync();
    if (rank == 0) {
        // Tile x belongs to part ((x + 1) P - 1) / N.
        const int c0 = static_cast<int>(((us + 1) * P - 1) / N), c1 = static_cast<int>(((us + ntiles) * P - 1) / N);
        const bool last = atomicAdd(p.counters + unit, 1) == c1 - c0;
        flag[0] = last ? c1 - c0 + 1 : 0;
        flag[1] = c0;
        if (last) p.counters[unit] = 0;  // ready for the next call
    }
    party.sync();
    const int n = flag[0];
    if (n > 0) {
        __threadfence();
        const float* base = p.partials + static_cast<size_t>(unit + flag[1]) * p.part_rows * PS;
        const size_t step = static_cast<size_t>(p.part_rows) * PS;
        for (int idx = rank; idx < kRows * C4; idx += party.threads()) {
            const int lr = idx / C4, c4 = idx - lr * C4;
            if (!((valid >> lr) & 1u)) continue;
            const float* row = base + static_cast<size_t>(lr) * PS;
            float M = -INFINITY, L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k0 = 0; k0 < n; k0 += kChunk) {
                float2 ml[kChunk];
                float4 o[kChunk];
#pragma unroll
                for (int k = 0; k < kChunk; ++k) {
                    const float* part = row + (k0 + k < n ? k0 + k : k0) * step;
                    ml[k] = __ldcg(reinterpret_cast<const float2*>(part + D));
                    o[k] = __ldcg(reinterpret_cast<const float4*>(part) + c4);
                    if (k0 + k >= n) ml[k] = make_float2(-INFINITY, 0.f);
                }
                const float old = M;
#pragma unroll
                for (int k = 0; k < kChunk; ++k) M = fmaxf(M, ml[k].x);
                const float Mu = M == -INFINITY ? 0.f : M;
                const float f = ptx::ex2(old - Mu);  // (0 before the first)
                L *= f;
                acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll
                for (int k = 0; k < kChunk; ++k) {
                    if (k0 + k >= n) break;
                    const float w = ptx::ex2(ml[k].x - Mu);
                    L = fmaf(w, ml[k].y, L);
                    acc.x = fmaf(w, o[k].x, acc.x);
                    acc.y = fmaf(w, o[k].y, acc.y);
                    acc.z = fmaf(w, o[k].z, acc.z);
                    acc.w = fmaf(w, o[k].w, acc.w);
                }
            }
            write_row<D>(p, row0 + lr, c4, acc, M, L, true, 0, lr);
        }
    }
}

// One producer warp: the tiles x0 .. x1 - 1 of its group (the party's first, then
// every step-th), a stage each, lanes 0 .. 3 issuing a tile's copies of K, V
// and their scale words side by side.
template <int D, int kStages, bool DP, int kGroups, bool kSplit>
__device__ __forceinline__ void produce(const DecodeParams& p, const Part<DP>& wp, int x0, int x1, const Party<kGroups, kSplit>& party,
                                        int lane, uint32_t stage0, uint32_t bar0, volatile int* abort_flag) {
    using St = Stage<D>;
    Cursor<DP, kKT> cur;
    cur.init(wp, x0);
    const bool is_v = (lane & 1) != 0, is_scale = (lane & 2) != 0;
    const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.v_cache : p.k_cache);
    const uint32_t* words = is_v ? p.q4.v : p.q4.k;
    const uint32_t dst_off = is_scale ? 2 * St::kCodeB + (is_v ? kKT * 4 : 0) : (is_v ? St::kCodeB : 0);
    const int step = party.step();
    int mine = party.first_tile(), stage = party.grp, phase = 1;  // (the first round of stages is free)
    int issued = 0;
    bool stop = false;
    for (int x = x0; x < x1 && !stop;) {
        const int b = cur.q / p.RB, kvh = cur.kvh;
        const int nseg = min(cur.nt - cur.j, x1 - x), it_end = x - x0 + nseg;
        int extent, min_lim;
        block_bounds(wp, b, cur.q - b * p.RB, extent, min_lim);
        const int first = (cur.t0 + cur.j) * kKT - (x - x0) * kKT;  // + it * kKT: the tile's first key
        // The tile's rows lie behind one another: one copy each of K, of V and
        // of their scale words, up to the last visible key (scale words to the
        // next multiple of 4, which the unit's stride holds).  The row of the
        // next tile is looked up before this one's stage is waited for.
        int row = mine < it_end ? key_row(p, b, kvh, first + mine * kKT) : 0;
        for (; mine < it_end; mine += step) {
            const int n = min(kKT, extent - (first + mine * kKT));
            const int next = mine + step < it_end ? key_row(p, b, kvh, first + (mine + step) * kKT) : 0;
            const uint32_t full = bar0 + 8 * stage;
            if (!ptx::mbar_try_wait(bar0 + 8 * (kStages + stage), phase) &&
                !ptx::mbar_wait_bounded(bar0 + 8 * (kStages + stage), phase, kWaitLimitNs)) {
                if (lane == 0) {
                    atomicExch(p.err, kDevTimeoutEmpty);
                    *abort_flag = 1;
                }
                stop = true;  // (a producer is in no named barrier, so it may stop early)
            }
            if (__any_sync(0xffffffffu, stop)) {
                stop = true;
                break;
            }
            const uint32_t cbytes = n * St::kRowB, sbytes = (n + 3) / 4 * 16;
            if (lane == 0) ptx::mbar_arrive_expect_tx(full, 2 * (cbytes + sbytes));
            __syncwarp();
            if (lane < 4)
                ptx::bulk_load(stage0 + stage * St::kBytes + dst_off,
                          is_scale ? static_cast<const void*>(words + q4::scale_index(p.q4, row))
                                   : static_cast<const void*>(src + static_cast<size_t>(row) * St::kRowB),
                          is_scale ? sbytes : cbytes, full);
            row = next;
            ++issued;
            stage += kGroups;
            if (stage >= kStages) {
                stage -= kStages;
                phase ^= 1;
            }
        }
        x += nseg;
        cur.j = cur.nt - 1;
        if (x < x1) cur.advance(wp);
    }
    // Never leave the CTA with copies in flight: wait (bounded) for the last
    // phase armed on each of this warp's stages (in a clean run they have
    // completed).
    constexpr int kOwn = kStages / kGroups;  // this warp's stages
    for (int i = max(0, issued - kOwn); i < issued; ++i) {
        const int st = party.grp + i % kOwn * kGroups;
        if (!ptx::mbar_wait_bounded(bar0 + 8 * st, (i / kOwn) & 1, kWaitLimitNs)) {
            if (lane == 0) atomicExch(p.err, kDevTimeoutDrain);
            break;
        }
    }
}

// The chunk's rows that fall into the 32 keys from key0 on (staged from row
// `koff` of the tile on) are quantised here, patched into the staged tile, whose
// copy of them is stale, and written to the cache.  Half a warp takes K and half
// V, eight values a lane.
template <int D>
__device__ __forceinline__ void append_slice(const DecodeParams& p, int b, int kvh, int prior, int nn, int key0, int koff,
                                             int lane, uint8_t* stage) {
    using St = Stage<D>;
    const int lo = max(prior, key0), hi = min(prior + nn, key0 + kWarpKeys);
    for (int pos = lo; pos < hi; ++pos) {
        const bool is_v = lane >= 16;
        const int c = lane & 15, r = pos - key0 + koff;
        const bool live = c < D / 8;
        const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.v_new : p.k_new) +
                             ((static_cast<size_t>(b) * p.Hkv + kvh) * p.Tn + (pos - prior)) * (D * 2);
        const uint4 val = live ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {val.x, val.y, val.z, val.w};
        uint32_t range = range8(w);
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) range = max2(range, __shfl_xor_sync(0xffffffffu, range, d));
        const RowScale sc = row_scale(range);
        const uint32_t code = encode8(w, sc);
        bool bad = false;
        const int row = phys_row(p.pg, p.ring, p.Hkv, p.max_len, b, kvh, pos, &bad);
        uint8_t* stg = stage + (is_v ? St::kCodeB : 0);
        uint8_t* words = stage + 2 * St::kCodeB + (is_v ? kKT * 4 : 0);
        if (live) {
            *reinterpret_cast<uint32_t*>(stg + r * St::kRowB + c * 4) = code;
            if (!bad)
                reinterpret_cast<uint32_t*>(is_v ? p.v_cache : p.k_cache)[static_cast<size_t>(row) * (D / 8) + c] =
                    code;
        }
        if (c == 0) {
            *reinterpret_cast<uint32_t*>(words + r * 4) = sc.word;
            if (!bad) (is_v ? p.q4.v : p.q4.k)[scale_index(p.q4, row)] = sc.word;
        }
    }
    if (lo < hi) {
        ptx::fence_proxy_async_smem();
        __syncwarp();
    }
}

}  // namespace q4
}  // namespace kvc
