// Split-KV GQA attention over a cache held in 4 bits (KVC_Q4), head widths 128
// and 64: decode, short verify, and any call cut into blocks of 8 or 16 query
// rows per KV head.  Semantics, work partition and the merge across CTAs are
// those of the bf16 split-KV kernel.
//
// The mathematics.  A stored row stands for s (c - z): one step s and zero
// point z a row, codes c = 0 .. 15.  With raw = q . c,
//   score = s_k (raw - z_k sum(q)) / sqrt(d)
//   out   = sum_k p_k s_v (c_k - z_v) / sum_k p_k
// so no single value is ever rescaled: K's step and zero point act on a score,
// V's step joins the softmax weight, and V's zero point is one running sum a
// query row.
//
// Codes as matrix operands.  A 4-bit integer in the low bits of an f16 is the
// subnormal c 2^-24, exactly, and at bits 4 .. 7 it is c 2^-20; the tensor core
// multiplies subnormals exactly.  So unpacking a word of eight codes into four
// f16 pairs is four ANDs and a shift, with no conversion and no subtraction;
// the two powers of two are taken out of q beforehand (K) and out of the
// result (V).
//
// Operands are laid out transposed: S^T = K q^T and O^T = V^T P^T, with the
// cache as the 16-row A operand and the query rows as the 8-column B operand.
// Decode has 1 to 8 query rows a KV head, so an 8-wide side wastes half of what
// the usual 16-row side would.  P^T goes from accumulator to B operand by one
// 8x8 register transpose a block.
//  * K: a thread's codes of a key are one aligned 16-byte (8-byte, d = 64)
//    piece of the row, all of them used; the head dimension is permuted to
//    match in q's fragments.
//  * V: a thread's output dims are one 8-byte (4-byte) piece of each key's row;
//    two keys' words are woven into f16 pairs by a byte permute.
//  * The 8 keys of a block are read in the order perm8, which puts K's accesses
//    on distinct shared-memory banks and V's at most two to a bank (d = 128).
//
// Range.  q is scaled by a power of two to just below 2^15 a row, so that f16
// holds it exactly whatever its size.  Weights are f16 too: p s_v 2^(133 - e),
// e the largest step exponent met so far (moved, with O, when a larger one
// appears), below 2^16 as p is below 2^8 (the reference maximum moves only
// past that) and s_v 2^(127 - e) below 2.  f16 keeps 11 bits of a weight; the
// zero point's sum uses the rounded weights, so the rounding acts on
// c - z and not on c.  Sums, maxima, l and O are fp32.
//
// Rows that a query must not see may hold anything: their scores, steps and
// weights are replaced, never multiplied.  Codes cannot be NaN, so V needs no
// clearing.
//
// How (GB300).  One persistent CTA per SM; tiles of 128 keys (2 x 8 KB of codes
// and 1 KB of scale words at d = 128) stream through bulk copies into a ring of stages;
// four warps share a tile, 32 keys each, and three groups of four (two with 16
// query rows) take tiles in turn.
// A unit's states meet in shared memory at its end, so a CTA leaves one
// partial a unit.
// Every wait is bounded in time; on expiry an error code is recorded.

#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "kvc_internal.h"
#include "ptx.cuh"
#include "q4.cuh"
#include "splitkv.cuh"

namespace kvc {

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kLazyRescale = 8.0f;  // log2 of the largest factor p may reach above the reference
constexpr int kKT = kQ4KeyTile;       // keys per tile
constexpr int kWarpKeys = 32;
constexpr uint32_t kMinExp = 6;       // 2^(133 - 6) is the largest power of two of an fp32
constexpr int kTileWarps = kKT / kWarpKeys;  // warps that share a tile

// D: head width; QB: blocks of 8 query rows.
template <int D, int QB>
struct Q4Shape {
    // Warp groups taking tiles in turn: as many as leave a thread the registers
    // it needs (128 with 12 consumer warps, 168 with 8).
    static constexpr int kGroups = QB == 1 ? 3 : 2;
    static constexpr int kCW = kGroups * kTileWarps;
    static constexpr int kCT = kCW * 32;
    static constexpr int kThreads = kCT + 32 * kGroups;  // a producer warp a group
    static constexpr int kRows = 8 * QB;
    static constexpr int kRowB = D / 2;            // bytes of a row's codes
    static constexpr int kCodeB = kKT * kRowB;     // one tile's K (or V) codes
    static constexpr int kStageB = 2 * kCodeB + 2 * kKT * 4;
    static constexpr int kPS = D + 4;              // floats of a state's row: O, m, l, pad
    static constexpr size_t kObuf = static_cast<size_t>(kCW) * kRows * kPS * sizeof(float);
    static constexpr int kFit = static_cast<int>((232448 - 1024 - 512 - kObuf) / kStageB);
    // A multiple of the groups, so that a stage belongs to one of them and a
    // stage's phases reach its warps in order.
    static constexpr int kStages = (kFit < 20 ? kFit : 20) / kGroups * kGroups;
    static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStageB + kObuf + 2 * kStages * 8 + 16;
    static_assert(kSmem <= 232448, "shared memory per CTA");
};

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
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t v) {
    __half2 h;
    memcpy(&h, &v, 4);
    return __half22float2(h);
}
// A small unsigned integer (below 2^16) as a float.
__device__ __forceinline__ float small_to_f32(uint32_t z) { return __uint_as_float(0x4B000000u | z) - 8388608.0f; }

// What a row block's queries see: one past the last visible key, and the
// smallest last key of a valid query.
template <bool DP>
__device__ __forceinline__ void block_bounds(const Part<DP>& w, int b, int rb, int& extent, int& min_lim) {
    const DecodeParams& p = w.p;
    const int prior = w.prior(b), nn = w.n_new(b);
    const int r0 = rb * p.RPB, r1 = min(p.R, r0 + p.RPB);
    extent = 0;
    min_lim = 0x7fffffff;
    for (int r = r0; r < r1; ++r) {
        const int t = r % p.T;
        if (t < nn) {
            min_lim = min(min_lim, prior + t);
            extent = max(extent, prior + t + 1);
        }
    }
}

// DP: the partition comes from a device plan; TREE: draft-tree ancestor masks.
template <int D, int QB, bool DP, bool TREE>
__global__ void __launch_bounds__(Q4Shape<D, QB>::kThreads, 1)
    decode_q4_kernel(const __grid_constant__ DecodeParams p) {
    using S = Q4Shape<D, QB>;
    constexpr int kStages = S::kStages;
    constexpr int PS = S::kPS;
    constexpr int KW = D / 32;   // 32-bit words of a thread's K codes a key (two MMA k-steps each)
    constexpr int VW = D / 64;   // 32-bit words of a thread's V codes a key (four 16-dim blocks each)
    constexpr int MB = D / 16;   // 16-dim blocks of O^T
    constexpr int KB = kWarpKeys / 16;  // 16-key blocks of a slice

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* obuf = reinterpret_cast<float*>(smem + static_cast<size_t>(kStages) * S::kStageB);  // [kCW][kRows][PS]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(kStages) * S::kStageB + S::kObuf);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * kStages);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Part<DP> wp{p};
    long long N = DP ? 0 : wp.total_tiles();
    const long long P = gridDim.x;
    int x0 = static_cast<int>(static_cast<long long>(blockIdx.x) * N / P);
    int x1 = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * N / P);

    const uint32_t stage0 = ptx::smem_addr(smem);
    const uint32_t bar0 = ptx::smem_addr(bars);  // full[s] = bar0 + 8s, empty[s] = bar0 + 8(kStages + s)
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(bar0 + 8 * s, 1);
            ptx::mbar_init(bar0 + 8 * (kStages + s), kTileWarps);
        }
        *abort_flag = 0;
        ptx::fence_barrier_init();
    }
    __syncthreads();
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (DP) {
        if (p.dplan->skip) return;  // a rejected device-resident step: nothing is written
        N = wp.total_tiles();
        x0 = static_cast<int>(static_cast<long long>(blockIdx.x) * N / P);
        x1 = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * N / P);
    }

    // Padded queries (t >= n_new[b]) output zeros; spread over the whole grid.
    {
        const int rows_total = p.B * p.Hq * p.T;
        for (int row = blockIdx.x * S::kThreads + tid; row < rows_total; row += gridDim.x * S::kThreads) {
            const int t = row % p.T;
            const int b = row / (p.Hq * p.T);
            if (t >= wp.n_new(b)) {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + static_cast<size_t>(row) * D);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }
    if (x0 >= x1) return;

    // ------------------------------------------------------------------ producers
    // One warp a group, so that the copies of consecutive tiles are issued side
    // by side; lanes 0 .. 3 issue a tile's copies of K, V and their scale words.
    if (warp >= S::kCW) {
        Cursor<DP, kKT> cur;
        cur.init(wp, x0);
        const bool is_v = (lane & 1) != 0, is_scale = (lane & 2) != 0;
        const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.v_cache : p.k_cache);
        const uint32_t* words = is_v ? p.q4.v : p.q4.k;
        const uint32_t dst_off = is_scale ? 2 * S::kCodeB + (is_v ? kKT * 4 : 0) : (is_v ? S::kCodeB : 0);
        int mine = warp - S::kCW, stage = mine, phase = 1;  // (the first round of stages is free)
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
            for (; mine < it_end; mine += S::kGroups) {
                const int n = min(kKT, extent - (first + mine * kKT));
                const int next = mine + S::kGroups < it_end ? key_row(p, b, kvh, first + (mine + S::kGroups) * kKT) : 0;
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
                const uint32_t cbytes = n * S::kRowB, sbytes = (n + 3) / 4 * 16;
                if (lane == 0) ptx::mbar_arrive_expect_tx(full, 2 * (cbytes + sbytes));
                __syncwarp();
                if (lane < 4)
                    ptx::bulk_load(stage0 + stage * S::kStageB + dst_off,
                              is_scale ? static_cast<const void*>(words + q4::scale_index(p.q4, row))
                                       : static_cast<const void*>(src + static_cast<size_t>(row) * S::kRowB),
                              is_scale ? sbytes : cbytes, full);
                row = next;
                ++issued;
                stage += S::kGroups;
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
        constexpr int kOwn = kStages / S::kGroups;  // this warp's stages
        for (int i = max(0, issued - kOwn); i < issued; ++i) {
            const int st = warp - S::kCW + i % kOwn * S::kGroups;
            if (!ptx::mbar_wait_bounded(bar0 + 8 * st, (i / kOwn) & 1, kWaitLimitNs)) {
                if (lane == 0) atomicExch(p.err, kDevTimeoutDrain);
                break;
            }
        }
        return;
    }

    // ------------------------------------------------------------------ consumers
    const int grp = warp / kTileWarps;                 // this warp's tiles: those of its group
    const int koff = (warp % kTileWarps) * kWarpKeys;  // its keys of a tile
    const int quad = lane & 3, g = lane >> 2;
    const int kg = perm8<D>(g);                                    // K: key of accumulator row g (and + 8)
    const int va = perm8<D>(2 * quad), vb = perm8<D>(2 * quad + 1);  // V: keys of the k index 2 quad, 2 quad + 1
    // Byte offsets of this thread's pieces in a tile.
    const uint32_t kpiece = (koff + kg) * S::kRowB + quad * (D / 8);
    const uint32_t vpiece_a = (koff + va) * S::kRowB + g * (D / 16);
    const uint32_t vpiece_b = (koff + vb) * S::kRowB + g * (D / 16);

    Cursor<DP, kKT> cur;
    cur.init(wp, x0);
    int mine = grp, stage = grp, phase = 0;  // this warp's next tile of the CTA's sequence, its stage and parity

    for (int x = x0; x < x1;) {
        // One segment: this CTA's tiles of one unit.
        const int b = cur.q / p.RB, rb = cur.q - b * p.RB, kvh = cur.kvh, j0 = cur.j;
        const int nseg = min(cur.nt - j0, x1 - x);
        const int it_end = x - x0 + nseg;
        const int prior = wp.prior(b), nn = wp.n_new(b);
        int extent, min_lim;
        block_bounds(wp, b, rb, extent, min_lim);
        const int max_lo = p.window > 0 ? extent - 1 - p.window : -1;  // keys > max_lo are in every query's window
        const int min_lo = p.window > 0 ? min_lim - p.window : -1;     // keys <= min_lo in none
        const int seg_key0 = (cur.t0 + j0) * kKT + koff - (x - x0) * kKT;  // + it * kKT: the slice's first key

        // Query fragments: this thread holds query row g's dims quad * D / 4 ..,
        // word by word; the k-steps of a word take its value pairs (0, 1), (2, 3)
        // and (4, 5), (6, 7), whose codes come as c 2^-24 and c 2^-20 in turn.
        // All rows are scaled by one power of two, 2^(141 - e), e the exponent
        // field of the largest |q|.
        uint32_t qa[QB][2 * KW][2];
        float qs[QB][2];   // sums of the scaled q of query rows 8 nb + 2 quad, + 1, times 2^-24
        float rs;          // scores' factor: 2^(e - 141) 2^24 log2(e) / sqrt(d)
        int lim[QB][2];    // last visible key (-1: no such query)
        {
            uint4 w[QB][KW];
            uint32_t top = 0;
#pragma unroll
            for (int nb = 0; nb < QB; ++nb) {
                const int r = rb * p.RPB + nb * 8 + g;
                const uint4* qrow = nullptr;
                if (r < p.R)
                    qrow = reinterpret_cast<const uint4*>(
                        static_cast<const __nv_bfloat16*>(p.q) +
                        ((static_cast<size_t>(b) * p.Hq + kvh * p.G + r / p.T) * p.T + r % p.T) * D + quad * (D / 4));
#pragma unroll
                for (int i = 0; i < KW; ++i) {
                    w[nb][i] = qrow ? __ldg(qrow + i) : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t u[4] = {w[nb][i].x, w[nb][i].y, w[nb][i].z, w[nb][i].w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) top = max(top, max(u[c] & 0x7FFFu, (u[c] >> 16) & 0x7FFFu));
                }
            }
            const int e = max(14, static_cast<int>(__reduce_max_sync(0xffffffffu, top) >> 7));
            const float f = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);
            rs = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(min(254, e + 10)) << 23);
#pragma unroll
            for (int nb = 0; nb < QB; ++nb) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < KW; ++i) {
                    const uint32_t u[4] = {w[nb][i].x, w[nb][i].y, w[nb][i].z, w[nb][i].w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float a0 = __uint_as_float(u[c] << 16) * f, a1 = __uint_as_float(u[c] & 0xFFFF0000u) * f;
                        sum += a0 + a1;
                        const float t = (c & 1) ? 0.0625f : 1.f;
                        qa[nb][2 * i + (c >> 1)][c & 1] = ptx::pack_f16x2(a0 * t, a1 * t);
                    }
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    qs[nb][h] = __shfl_sync(0xffffffffu, sum, (2 * quad + h) * 4) * 5.9604644775390625e-8f;  // 2^-24
                    const int r = rb * p.RPB + nb * 8 + 2 * quad + h, t = r % p.T;
                    lim[nb][h] = (r < p.R && t < nn) ? prior + t : -1;
                }
            }
        }

        // The segment's state.
        float o[QB][MB][4];
        float m[QB][2], nm[QB][2], l[QB][2], zs[QB][2];  // rows' maximum (and its negative, 0 before any), sums of p, of p s_v z_v
        uint32_t vexp = kMinExp;                          // exponent field of the largest V step met (at least kMinExp)
        float vmul = __uint_as_float((260u - kMinExp) << 23);  // 2^(133 - vexp)
#pragma unroll
        for (int nb = 0; nb < QB; ++nb) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                m[nb][h] = -INFINITY;
                nm[nb][h] = l[nb][h] = zs[nb][h] = 0.f;
            }
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) o[nb][mb][0] = o[nb][mb][1] = o[nb][mb][2] = o[nb][mb][3] = 0.f;
        }

        // One slice of kWarpKeys keys from key0 on, staged at sK / sV / sS.
        // FULL: every valid query of the block sees every key of it.
        auto attend = [&](auto full_tag, const int key0, const uint32_t sK, const uint32_t sV, const uint32_t sS) {
            constexpr bool FULL = decltype(full_tag)::value;
            // S^T = K q^T: blocks of 16 keys x 8 query rows.
            float sc[KB][QB][4];
            uint32_t kw[KB][2], vw[KB][2];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    kw[kb][h] = lds32(sS + (koff + kb * 16 + kg + 8 * h) * 4);
                    vw[kb][h] = lds32(sS + (kKT + koff + kb * 16 + kg + 8 * h) * 4);
                }
                uint32_t k0w[KW], k1w[KW];
                const uint32_t ka = sK + kpiece + kb * 16 * S::kRowB;
                if constexpr (D == 128) {
                    const uint4 u = ptx::ld_shared_v4(ka), v = ptx::ld_shared_v4(ka + 8 * S::kRowB);
                    k0w[0] = u.x, k0w[1] = u.y, k0w[2] = u.z, k0w[3] = u.w;
                    k1w[0] = v.x, k1w[1] = v.y, k1w[2] = v.z, k1w[3] = v.w;
                } else {
                    const uint2 u = lds64(ka), v = lds64(ka + 8 * S::kRowB);
                    k0w[0] = u.x, k0w[1] = u.y;
                    k1w[0] = v.x, k1w[1] = v.y;
                }
#pragma unroll
                for (int nb = 0; nb < QB; ++nb) sc[kb][nb][0] = sc[kb][nb][1] = sc[kb][nb][2] = sc[kb][nb][3] = 0.f;
#pragma unroll
                for (int i = 0; i < KW; ++i) {
                    const uint32_t x0w = k0w[i], x1w = k1w[i], y0w = x0w >> 8, y1w = x1w >> 8;
                    const uint32_t a[4] = {x0w & 0x000F000Fu, x1w & 0x000F000Fu, x0w & 0x00F000F0u, x1w & 0x00F000F0u};
                    const uint32_t c[4] = {y0w & 0x000F000Fu, y1w & 0x000F000Fu, y0w & 0x00F000F0u, y1w & 0x00F000F0u};
#pragma unroll
                    for (int nb = 0; nb < QB; ++nb) {
                        ptx::mma_f16_16816(sc[kb][nb], a, qa[nb][2 * i][0], qa[nb][2 * i][1]);
                        ptx::mma_f16_16816(sc[kb][nb], c, qa[nb][2 * i + 1][0], qa[nb][2 * i + 1][1]);
                    }
                }
            }
            // Scores in base 2, masked; each row's maximum over the slice.  Keys
            // that no query of the block sees get no step, so that neither a
            // stale word nor its exponent enters.
            float mx[QB][2];
#pragma unroll
            for (int nb = 0; nb < QB; ++nb) mx[nb][0] = mx[nb][1] = -INFINITY;
            uint32_t ve = 0;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int key = key0 + kb * 16 + kg + 8 * h;
                    if (!FULL && (key >= extent || key <= min_lo)) kw[kb][h] = vw[kb][h] = 0u;
                    const uint32_t ex = vw[kb][h] >> 23;
                    ve = max(ve, ex == 255u ? 0u : ex);  // (a NaN step stays NaN under any factor)
                    const float ks = q4::step_of(kw[kb][h]) * rs, kz = -small_to_f32(kw[kb][h] & 0xFFFFu);
#pragma unroll
                    for (int nb = 0; nb < QB; ++nb)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float& v = sc[kb][nb][2 * h + c];
                            v = fmaf(kz, qs[nb][c], v) * ks;
                            if (!FULL) {
                                const int li = lim[nb][c];
                                bool see = key <= li && (p.window <= 0 || key > li - p.window);
                                if (TREE && see && key >= prior) see = (p.anc[b * p.T + (li - prior)] >> (key - prior)) & 1ull;
                                if (!see) v = -INFINITY;
                            }
                            mx[nb][c] = fmaxf(mx[nb][c], v);
                        }
                }
            }
            // (Each thread compares its own keys' maxima; they are joined only when
            // some row's reference has to move.)
            bool move = ve > vexp;
#pragma unroll
            for (int nb = 0; nb < QB; ++nb) move |= mx[nb][0] > m[nb][0] + kLazyRescale || mx[nb][1] > m[nb][1] + kLazyRescale;
            if (__any_sync(0xffffffffu, move)) {
                // Move the references; O, l and the zero points' sum follow.
                ve = max(vexp, __reduce_max_sync(0xffffffffu, ve));
                const float fv =
                    __uint_as_float(static_cast<uint32_t>(max(0, 127 + static_cast<int>(vexp) - static_cast<int>(ve))) << 23);
                vexp = ve;
                vmul = __uint_as_float((260u - vexp) << 23);
#pragma unroll
                for (int nb = 0; nb < QB; ++nb) {
                    float f[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) mx[nb][c] = fmaxf(mx[nb][c], __shfl_xor_sync(0xffffffffu, mx[nb][c], d));
                        const bool mv = mx[nb][c] > m[nb][c] + kLazyRescale;
                        const float al = !mv ? 1.f : (m[nb][c] == -INFINITY) ? 0.f : ptx::ex2(m[nb][c] - mx[nb][c]);
                        if (mv) {
                            m[nb][c] = mx[nb][c];
                            nm[nb][c] = -mx[nb][c];
                        }
                        l[nb][c] *= al;
                        f[c] = al * fv;
                        zs[nb][c] *= f[c];
                    }
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb) {
                        o[nb][mb][0] *= f[0];
                        o[nb][mb][1] *= f[1];
                        o[nb][mb][2] *= f[0];
                        o[nb][mb][3] *= f[1];
                    }
                }
            }
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                // Weights: p into l, p s_v (f16) into the products, times z_v into
                // the zero points' sum.
                const float vs0 = q4::step_of(vw[kb][0]) * vmul, vs1 = q4::step_of(vw[kb][1]) * vmul;
                const float vz0 = small_to_f32(vw[kb][0] & 0xFFFFu), vz1 = small_to_f32(vw[kb][1] & 0xFFFFu);
                uint32_t pb[QB][2];
#pragma unroll
                for (int nb = 0; nb < QB; ++nb) {
                    float pw[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v = sc[kb][nb][e], pe = ptx::ex2(v + nm[nb][e & 1]);
                        l[nb][e & 1] += pe;
                        pw[e] = pe * ((e < 2) ? vs0 : vs1);
                        if (!FULL && v == -INFINITY) pw[e] = 0.f;  // (a NaN step that this query does not see)
                    }
                    const uint32_t h0 = ptx::pack_f16x2(pw[0], pw[1]), h1 = ptx::pack_f16x2(pw[2], pw[3]);
                    const float2 r0 = f16x2_to_f32(h0), r1 = f16x2_to_f32(h1);
                    zs[nb][0] = fmaf(r1.x, vz1, fmaf(r0.x, vz0, zs[nb][0]));
                    zs[nb][1] = fmaf(r1.y, vz1, fmaf(r0.y, vz0, zs[nb][1]));
                    pb[nb][0] = transpose8x8(h0);
                    pb[nb][1] = transpose8x8(h1);
                }
                // O^T += V^T P^T.
                uint32_t va0[VW], vb0[VW], va8[VW], vb8[VW];
                const uint32_t pa = sV + vpiece_a + kb * 16 * S::kRowB, pc = sV + vpiece_b + kb * 16 * S::kRowB;
                if constexpr (D == 128) {
                    const uint2 t0 = lds64(pa), t1 = lds64(pc);
                    const uint2 t2 = lds64(pa + 8 * S::kRowB), t3 = lds64(pc + 8 * S::kRowB);
                    va0[0] = t0.x, va0[1] = t0.y, vb0[0] = t1.x, vb0[1] = t1.y;
                    va8[0] = t2.x, va8[1] = t2.y, vb8[0] = t3.x, vb8[1] = t3.y;
                } else {
                    va0[0] = lds32(pa), vb0[0] = lds32(pc);
                    va8[0] = lds32(pa + 8 * S::kRowB), vb8[0] = lds32(pc + 8 * S::kRowB);
                }
#pragma unroll
                for (int i = 0; i < VW; ++i) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // even, then odd values of the word
                        const uint32_t sel = h ? 0x7632u : 0x5410u;
                        const uint32_t u = ptx::prmt(va0[i], vb0[i], sel), v = ptx::prmt(va8[i], vb8[i], sel);
                        const uint32_t u8 = u >> 8, v8 = v >> 8;
                        const uint32_t a[4] = {u & 0x000F000Fu, u & 0x00F000F0u, v & 0x000F000Fu, v & 0x00F000F0u};
                        const uint32_t c[4] = {u8 & 0x000F000Fu, u8 & 0x00F000F0u, v8 & 0x000F000Fu, v8 & 0x00F000F0u};
#pragma unroll
                        for (int nb = 0; nb < QB; ++nb) {
                            ptx::mma_f16_16816(o[nb][4 * i + 2 * h], a, pb[nb][0], pb[nb][1]);
                            ptx::mma_f16_16816(o[nb][4 * i + 2 * h + 1], c, pb[nb][0], pb[nb][1]);
                        }
                    }
                }
            }
        };

        for (; mine < it_end; mine += S::kGroups) {
            // On expiry the warp records the error and carries on with whatever
            // the stage holds (the call's output is then invalid): consumer
            // warps meet at named barriers, so none may leave the loop alone.
            if (!ptx::mbar_try_wait(bar0 + 8 * stage, phase) &&
                !ptx::mbar_wait_bounded(bar0 + 8 * stage, phase, *abort_flag ? 0ull : kWaitLimitNs)) {
                atomicExch(p.err, kDevTimeoutFull);
                *abort_flag = 1;
            }
            const uint32_t sK = stage0 + stage * S::kStageB, sV = sK + S::kCodeB, sS = sV + S::kCodeB;
            const int key0 = seg_key0 + mine * kKT;

            if (p.append_new && key0 + kWarpKeys > prior) {
                // In-kernel append: the chunk's rows that fall into this slice are
                // quantised here, patched into the staged tile (whose copy of
                // them is stale) and written to the cache.  Half a warp takes K
                // and half V, eight values a lane.
                const int lo = max(prior, key0), hi = min(prior + nn, key0 + kWarpKeys);
                for (int pos = lo; pos < hi; ++pos) {
                    const bool is_v = lane >= 16;
                    const int c = lane & 15, r = pos - key0 + koff;
                    const bool live = c < D / 8;
                    const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.v_new : p.k_new) +
                                         ((static_cast<size_t>(b) * p.Hkv + kvh) * p.Tn + (pos - prior)) * (D * 2);
                    const uint4 val = live ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t w[4] = {val.x, val.y, val.z, val.w};
                    uint32_t range = q4::range8(w);
#pragma unroll
                    for (int d = 8; d > 0; d >>= 1) range = q4::max2(range, __shfl_xor_sync(0xffffffffu, range, d));
                    const q4::RowScale sc = q4::row_scale(range);
                    const uint32_t code = q4::encode8(w, sc);
                    bool bad = false;
                    const int row = phys_row(p.pg, p.ring, p.Hkv, p.max_len, b, kvh, pos, &bad);
                    uint8_t* stg = smem + stage * S::kStageB + (is_v ? S::kCodeB : 0);
                    uint8_t* words = smem + stage * S::kStageB + 2 * S::kCodeB + (is_v ? kKT * 4 : 0);
                    if (live) {
                        *reinterpret_cast<uint32_t*>(stg + r * S::kRowB + c * 4) = code;
                        if (!bad)
                            reinterpret_cast<uint32_t*>(is_v ? p.v_cache : p.k_cache)[static_cast<size_t>(row) * (D / 8) + c] =
                                code;
                    }
                    if (c == 0) {
                        *reinterpret_cast<uint32_t*>(words + r * 4) = sc.word;
                        if (!bad) (is_v ? p.q4.v : p.q4.k)[q4::scale_index(p.q4, row)] = sc.word;
                    }
                }
                if (lo < hi) {
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                }
            }

            if (key0 + kWarpKeys - 1 <= min_lim && key0 > max_lo && (!TREE || key0 + kWarpKeys <= prior))
                attend(std::true_type(), key0, sK, sV, sS);
            else if (key0 < extent && key0 + kWarpKeys - 1 > min_lo)
                attend(std::false_type(), key0, sK, sV, sS);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar0 + 8 * (kStages + stage));
            stage += S::kGroups;
            if (stage >= kStages) {
                stage -= kStages;
                phase ^= 1;
            }
        }

        // The segment's end: every warp's state of every query row into shared
        // memory, O in real units.
        {
#pragma unroll
            for (int nb = 0; nb < QB; ++nb)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        l[nb][h] += __shfl_xor_sync(0xffffffffu, l[nb][h], d);
                        zs[nb][h] += __shfl_xor_sync(0xffffffffu, zs[nb][h], d);
                    }
                    // A row whose every score is NaN keeps that through the merges.
                    if (m[nb][h] == -INFINITY && l[nb][h] != 0.f) m[nb][h] = 0.f;
                    const int lr = nb * 8 + 2 * quad + h;
                    float* st = obuf + (warp * S::kRows + lr) * PS;
                    const float real = __uint_as_float(vexp << 23);  // 2^(vexp - 127)
#pragma unroll
                    for (int i = 0; i < VW; ++i) {
                        // values 0 .. 7 of word i: blocks 4i .. 4i+3 hold (0, 2), (4, 6), (1, 3), (5, 7)
                        float e[8];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int v = (c & 1) * 4 + (c >> 1);
                            e[v] = fmaf(o[nb][4 * i + c][h], 16777216.f, -zs[nb][h]) * 0.015625f * real;
                            e[v + 2] = fmaf(o[nb][4 * i + c][2 + h], 1048576.f, -zs[nb][h]) * 0.015625f * real;
                        }
                        float4* d4 = reinterpret_cast<float4*>(st + g * (D / 8) + i * 8);
                        d4[0] = make_float4(e[0], e[1], e[2], e[3]);
                        d4[1] = make_float4(e[4], e[5], e[6], e[7]);
                    }
                    if (g == 0) {
                        st[D] = m[nb][h];
                        st[D + 1] = l[nb][h];
                    }
                }
            ptx::named_barrier_sync(1, S::kCT);
            // Merge them in the order of the warps, and write the unit's output
            // (this CTA saw all of it) or the CTA's partial.
            const bool sole = nseg == cur.nt;
            constexpr int C4 = D / 4;
            for (int idx = tid; idx < S::kRows * C4; idx += S::kCT) {
                const int lr = idx / C4, c4 = idx - lr * C4;
                const int r = rb * p.RPB + lr;
                if (r >= p.R) continue;
                const int t = r % p.T;
                if (t >= nn) continue;
                const float* st = obuf + lr * PS;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < S::kCW; ++w) M = fmaxf(M, st[w * S::kRows * PS + D]);
                const float Mu = M == -INFINITY ? 0.f : M;
                float L = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < S::kCW; ++w) {
                    const float* sw = st + w * S::kRows * PS;
                    const float f = ptx::ex2(sw[D] - Mu);
                    const float4 v = reinterpret_cast<const float4*>(sw)[c4];
                    L = fmaf(sw[D + 1], f, L);
                    acc.x = fmaf(v.x, f, acc.x);
                    acc.y = fmaf(v.y, f, acc.y);
                    acc.z = fmaf(v.z, f, acc.z);
                    acc.w = fmaf(v.w, f, acc.w);
                }
                if (sole) {
                    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // (NaN stays)
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) +
                                         ((static_cast<size_t>(b) * p.Hq + kvh * p.G + r / p.T) * p.T + t) * D + c4 * 4;
                    uint2 v;
                    v.x = ptx::pack_bf16x2(acc.x * inv, acc.y * inv);
                    v.y = ptx::pack_bf16x2(acc.z * inv, acc.w * inv);
                    *reinterpret_cast<uint2*>(dst) = v;
                } else {
                    const int slot = cur.q * p.Hkv + kvh + blockIdx.x;
                    float* part = p.partials + (static_cast<size_t>(slot) * p.part_rows + lr) * PS;
                    reinterpret_cast<float4*>(part)[c4] = acc;
                    if (c4 == 0) {
                        part[D] = M;
                        part[D + 1] = L;
                    }
                }
            }
            ptx::named_barrier_sync(1, S::kCT);
        }
        x += nseg;
        cur.j = cur.nt - 1;  // (the next unit; past the last one nothing reads it)
        if (x < x1) cur.advance(wp);
    }
}

template <int D, int QB, bool DP, bool TREE>
cudaError_t launch_q4_t(const DecodeParams& p, int grid, cudaStream_t stream) {
    using S = Q4Shape<D, QB>;
    static bool attr_set = false;
    if (!attr_set) {
        cudaError_t e = cudaFuncSetAttribute(decode_q4_kernel<D, QB, DP, TREE>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
        if (e != cudaSuccess) return e;
        attr_set = true;
    }
    cudaError_t e = launch_pdl(decode_q4_kernel<D, QB, DP, TREE>, dim3(grid), dim3(S::kThreads), S::kSmem, stream, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <int D, int QB>
cudaError_t launch_q4_shape(const DecodeParams& p, int grid, cudaStream_t stream) {
    if (p.dplan) return p.anc ? cudaErrorInvalidValue : launch_q4_t<D, QB, true, false>(p, grid, stream);
    return p.anc ? launch_q4_t<D, QB, false, true>(p, grid, stream) : launch_q4_t<D, QB, false, false>(p, grid, stream);
}

}  // namespace

cudaError_t launch_decode_q4(const DecodeParams& p, int grid, int d, cudaStream_t stream) {
    if (p.RPB != 8 && p.RPB != 16) return cudaErrorInvalidValue;
    if (d == 128)
        return p.RPB == 8 ? launch_q4_shape<128, 1>(p, grid, stream) : launch_q4_shape<128, 2>(p, grid, stream);
    if (d == 64)
        return p.RPB == 8 ? launch_q4_shape<64, 1>(p, grid, stream) : launch_q4_shape<64, 2>(p, grid, stream);
    return cudaErrorInvalidValue;
}

}  // namespace kvc
