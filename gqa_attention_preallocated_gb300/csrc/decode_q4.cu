// Split-KV GQA attention over a cache held in 4 bits (KVC_Q4): up to 8 query
// rows per KV head at head width 128 (decode; more rows in decode_q4_wide.cu),
// up to 32, and any number in blocks of 32, at head width 64.  Semantics and work
// partition are those of the bf16 split-KV kernel.
//
// The mathematics.  A stored row stands for s (c - z): one step s and zero
// point z a row, codes c = 0 .. 15.  With raw = q . c,
//   score = s_k (raw - z_k sum(q)) / sqrt(d)
//   out   = sum_k p_k s_v (c_k - z_v) / sum_k p_k
// so no single value is ever rescaled: K's step and zero point act on a score,
// V's step joins the softmax weight, and V's zero points are one more dimension
// of the output, which is taken from all the others at the end.
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
// holds it exactly whatever its size (below 2^112, where the factor that undoes
// it leaves fp32).  Weights are f16 too: p s_v 2^(133 - e),
// e the largest step exponent met so far (moved, with O, when a larger one
// appears), below 2^16 as p is below 2^8 (the reference maximum moves only
// past that) and s_v 2^(127 - e) below 2.  f16 keeps 11 bits of a weight, or
// 2^-31 of the largest step where that is more.  The zero points' sum runs
// through the same products as the codes' (their f16 pairs as one more row of
// V^T), so that the weights' rounding acts on c - z, and the tensor core's
// truncation, 2^-23 of a sum each time it adds, on both alike: over 131072 keys
// the two sums are some 300 times their difference.  Maxima, l and O are fp32.
//
// Rows that a query must not see may hold anything: their scores, steps and
// weights are replaced, never multiplied.  Codes cannot be NaN, so V needs no
// clearing.
//
// How (GB300).  One persistent CTA per SM; tiles of 128 keys (2 x 8 KB of codes
// and 1 KB of scale words at d = 128) stream through bulk copies into a ring of stages;
// four warps share a tile, 32 keys each.  Three groups of four (two with more
// than 16 query rows) take a unit's tiles in turn, and their states meet in
// shared memory at its end, so a CTA leaves one partial a unit; or, with many
// units, each group has a share of the tiles to itself (Party).  The last to
// leave a unit's partial merges them.
//
// Measured: 4 rows of 131072 tokens, 8 KV heads of 4 query rows, d = 128 (571 MB):
// 101 us, 5.7 TB/s; d = 64 (302 MB): 72 us, 4.2 TB/s; 32 rows of 6144: 46 us,
// 4.6 TB/s.  Bound by issue and its waits: a third of the issue slots used, 18 %
// of the tensor pipe, no warp's chain short enough to fill the rest.  Steps on the
// way, for the first: 288 us with 16 keys a warp and a copy a row, 181 with 32,
// 149 with untiled copies of whole tiles, 104 with a producer warp a group, 99
// without divisions in the address walk.
// Every wait is bounded in time; on expiry an error code is recorded.

#include <type_traits>

#include "q4_splitkv.cuh"

namespace kvc {

namespace {

using namespace q4;

// D: head width; QB: blocks of 8 query rows.
template <int D, int QB>
struct Q4Shape {
    // Warp groups taking tiles in turn: as many as leave a thread the registers
    // it needs (128 with 12 consumer warps, 168 with 8).
    static constexpr int kGroups = q4_groups(D, 8 * QB);
    static constexpr int kCW = kGroups * kTileWarps;
    static constexpr int kCT = kCW * 32;
    static constexpr int kThreads = kCT + 32 * kGroups;  // a producer warp a group
    static constexpr int kRows = 8 * QB;
    static constexpr int kRowB = Stage<D>::kRowB, kCodeB = Stage<D>::kCodeB, kStageB = Stage<D>::kBytes;
    static constexpr int kPS = D + 4;              // floats of a state's row: O, m, l, pad
    static constexpr size_t kObuf = static_cast<size_t>(kCW) * kRows * kPS * sizeof(float);
    static constexpr bool kQSmem = QB > 2;  // query fragments in shared memory, not in registers
    static constexpr size_t kQgroup = kQSmem ? QB * (D / 32) * 32 * 16 : 0, kQbuf = kGroups * kQgroup;
    static constexpr int kFit = static_cast<int>((232448 - 1024 - 512 - kQbuf - kObuf) / kStageB);
    // A multiple of the groups, so that a stage belongs to one of them and a
    // stage's phases reach its warps in order.
    static constexpr int kStages = (kFit < 20 ? kFit : 20) / kGroups * kGroups;
    static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStageB + kObuf + kQbuf + 2 * kStages * 8 + 16 + kGroups * sizeof(Segment);
    static_assert(kStages >= 2 * kGroups, "a stage to read and one to fill for every group");
    static_assert(kSmem <= 232448 && kGroups == q4_groups(D, kRows), "shared memory per CTA");
};

// DP: the partition comes from a device plan; TREE: draft-tree ancestor masks.
template <int D, int QB, bool DP, bool TREE, bool SPLIT>
__global__ void __launch_bounds__(Q4Shape<D, QB>::kThreads, 1)
    decode_q4_kernel(const __grid_constant__ DecodeParams p) {
    using S = Q4Shape<D, QB>;
    constexpr int kStages = S::kStages;
    constexpr int PS = S::kPS;
    constexpr int KW = D / 32;   // 32-bit words of a thread's K codes a key (two MMA k-steps each)
    constexpr int VW = D / 64;   // 32-bit words of a thread's V codes a key (four 16-dim blocks each)
    constexpr int MB = D / 16;   // 16-dim blocks of O^T
    // 16-key blocks taken together: both of a slice with one block of query rows
    // (two chains hide each other), one at a time with more (registers).
    constexpr int KB = QB == 1 ? 2 : 1;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* obuf = reinterpret_cast<float*>(smem + static_cast<size_t>(kStages) * S::kStageB);  // [kCW][kRows][PS]
    uint8_t* qbuf = smem + static_cast<size_t>(kStages) * S::kStageB + S::kObuf;
    const uint32_t qfrag = ptx::smem_addr(qbuf);
    uint64_t* bars = reinterpret_cast<uint64_t*>(qbuf + S::kQbuf);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * kStages);
    volatile Segment* segs = reinterpret_cast<volatile Segment*>(bars + 2 * kStages + 2);  // a group's

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Part<DP> wp{p};

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
    if (DP && p.dplan->skip) return;  // a rejected device-resident step: nothing is written

    zero_padded_queries<D, DP>(p, wp, tid, S::kThreads);
    const int grp = warp < S::kCW ? warp / kTileWarps : warp - S::kCW;
    const Party<S::kGroups, SPLIT> party{grp};
    int x0, x1;  // this party's tiles
    {
        const long long N = wp.total_tiles(), P = shares(wp), i = party.part();
        x0 = static_cast<int>(min(i, P) * N / P), x1 = static_cast<int>(min(i + 1, P) * N / P);
    }
    if (x0 >= x1) return;

    if (warp >= S::kCW) {
        produce<D, kStages, DP>(p, wp, x0, x1, party, lane, stage0, bar0, abort_flag);
        return;
    }

    // ------------------------------------------------------------------ consumers
    const int koff = (warp % kTileWarps) * kWarpKeys;  // its keys of a tile
    const int quad = lane & 3, g = lane >> 2;
    const int kg = perm8<D>(g);                                    // K: key of accumulator row g (and + 8)
    const int va = perm8<D>(2 * quad), vb = perm8<D>(2 * quad + 1);  // V: keys of the k index 2 quad, 2 quad + 1
    // Byte offsets of this thread's pieces in a tile.
    const uint32_t kpiece = kg * S::kRowB + quad * (D / 8);
    const uint32_t vpiece_a = va * S::kRowB + g * (D / 16);
    const uint32_t vpiece_b = vb * S::kRowB + g * (D / 16);

    Cursor<DP, kKT> cur;
    cur.init(wp, x0);
    volatile Segment* seg = segs + grp;
    int mine = party.first_tile(), stage = grp, phase = 0;  // this warp's next tile of the CTA's sequence, its stage and parity

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
        // Query row i of the block is row row0 + i of q and out (packed g * T + t);
        // lane i holds its last visible key (-1: no such query), `valid` has its bit.
        // (Kept in shared memory for the segment's end: registers are short.)
        const size_t row0 = (static_cast<size_t>(b) * p.Hq + kvh * p.G) * p.T + rb * p.RPB;
        int lane_lim;
        {
            const int r = rb * p.RPB + lane, t = r % p.T;
            lane_lim = (lane < S::kRows && r < p.R && t < nn) ? prior + t : -1;
        }
        const uint32_t valid = __ballot_sync(0xffffffffu, lane_lim >= 0);
        if ((tid & 127) == 0) {
            seg->row0 = row0;
            seg->valid = valid;
            seg->unit_tile = x - j0;
            seg->unit = cur.q * p.Hkv + kvh;
        }

        // Query fragments: this thread holds query row g's dims quad * D / 4 ..,
        // word by word; the k-steps of a word take its value pairs (0, 1), (2, 3)
        // and (4, 5), (6, 7), whose codes come as c 2^-24 and c 2^-20 in turn.
        // Each row is scaled by a power of two, 2^(141 - e), e the exponent field of
        // its largest |q|.
        uint4 qa[QB][KW];  // (in shared memory with many rows)
        float qs[QB][2];   // sums of the scaled q of query rows 8 nb + 2 quad, + 1, times 2^-24
        float rs[QB][2];   // their scores' factor: 2^(e - 141) 2^24 log2(e) / sqrt(d)
        {
#pragma unroll
            for (int nb = 0; nb < QB; ++nb) {
                const uint4* qrow = nullptr;
                if ((valid >> (nb * 8 + g)) & 1u)
                    qrow = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (row0 + nb * 8 + g) * D + quad * (D / 4));
                uint4 w[KW];
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < KW; ++i) {
                    w[i] = qrow ? __ldg(qrow + i) : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) top = max(top, max(u[c] & 0x7FFFu, (u[c] >> 16) & 0x7FFFu));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = max(14, static_cast<int>(top >> 7));
                const float f = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);
                const float rowf = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(min(254, e + 10)) << 23);
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < KW; ++i) {
                    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                    uint32_t hq[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float a0 = __uint_as_float(u[c] << 16) * f, a1 = __uint_as_float(u[c] & 0xFFFF0000u) * f;
                        sum += a0 + a1;
                        const float t = (c & 1) ? 0.0625f : 1.f;
                        hq[c] = ptx::pack_f16x2(a0 * t, a1 * t);
                    }
                    qa[nb][i] = make_uint4(hq[0], hq[1], hq[2], hq[3]);
                    if constexpr (S::kQSmem) {
                        if (warp % kTileWarps == nb) *reinterpret_cast<uint4*>(qbuf + grp * S::kQgroup + ((nb * KW + i) * 32 + lane) * 16) = qa[nb][i];
                    }
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    qs[nb][h] = __shfl_sync(0xffffffffu, sum, (2 * quad + h) * 4) * 5.9604644775390625e-8f;  // 2^-24
                    rs[nb][h] = __shfl_sync(0xffffffffu, rowf, (2 * quad + h) * 4);
                }
            }
        }

        if constexpr (S::kQSmem) ptx::named_barrier_sync(2 + grp, 128);

        // The segment's state.
        float o[QB][MB][4];
        // Rows' reference (and its negative, 0 before the first key; a row that is
        // no query keeps reference 0), sums of p; of p s_v z_v (the accumulator of
        // 16 equal rows).
        float m[QB][2], nm[QB][2], l[QB][2], zs[QB][4];
        bool fresh = true;                                // some query of the block has met no key yet
        uint32_t vexp = kMinExp;                          // exponent field of the largest V step met (at least kMinExp)
        float vmul = __uint_as_float((260u - kMinExp) << 23);  // 2^(133 - vexp)
#pragma unroll
        for (int nb = 0; nb < QB; ++nb) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                m[nb][h] = ((valid >> (nb * 8 + 2 * quad + h)) & 1u) ? -INFINITY : 0.f;
                nm[nb][h] = l[nb][h] = zs[nb][h] = zs[nb][2 + h] = 0.f;
            }
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) o[nb][mb][0] = o[nb][mb][1] = o[nb][mb][2] = o[nb][mb][3] = 0.f;
        }

        // KB blocks of 16 keys of this warp's slice, the first key at key0 and
        // row `at` of the tile staged at sK / sV / sS.  full: every valid query
        // of the block sees every key of them (a copy of the code without masks:
        // branches around them cost 4 % of a long decode).
        auto attend = [&](auto full_tag, const int key0, const int at, const uint32_t sK, const uint32_t sV, const uint32_t sS) {
            constexpr bool full = decltype(full_tag)::value;
            // S^T = K q^T: blocks of 16 keys x 8 query rows.
            float sc[KB][QB][4];
            uint32_t kw[KB][2], vw[KB][2];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    kw[kb][h] = lds32(sS + (at + kb * 16 + kg + 8 * h) * 4);
                    vw[kb][h] = lds32(sS + (kKT + at + kb * 16 + kg + 8 * h) * 4);
                }
                uint32_t k0w[KW], k1w[KW];
                const uint32_t ka = sK + kpiece + (at + kb * 16) * S::kRowB;
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
                        if constexpr (S::kQSmem) {
                            const uint4 f = ptx::ld_shared_v4(qfrag + grp * S::kQgroup + ((nb * KW + i) * 32 + lane) * 16);
                            ptx::mma_f16_16816(sc[kb][nb], a, f.x, f.y);
                            ptx::mma_f16_16816(sc[kb][nb], c, f.z, f.w);
                        } else {
                            ptx::mma_f16_16816(sc[kb][nb], a, qa[nb][i].x, qa[nb][i].y);
                            ptx::mma_f16_16816(sc[kb][nb], c, qa[nb][i].z, qa[nb][i].w);
                        }
                    }
                }
            }
            // Scores in base 2 less the row's reference, masked.  Keys that no
            // query of the block sees get no step, so that neither a stale word
            // nor its exponent enters.  The references move when one of them is
            // passed by more than kLazyRescale, V's exponent when a larger one
            // comes, and at a valid row's first key (fresh).
            if (!full) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int key = key0 + kb * 16 + kg + 8 * h;
                        if (key >= extent || key <= min_lo) kw[kb][h] = vw[kb][h] = 0u;
                    }
            }
            uint32_t ve = 0;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t ex = vw[kb][h] >> 23;
                    ve = max(ve, ex == 255u ? 0u : ex);  // (a NaN step stays NaN under any factor)
                    const float ks = q4::step_of(kw[kb][h]), kz = -zero_f32(kw[kb][h]);
#pragma unroll
                    for (int nb = 0; nb < QB; ++nb)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float& v = sc[kb][nb][2 * h + c];
                            v = fmaf(fmaf(kz, qs[nb][c], v), ks * rs[nb][c], nm[nb][c]);
                        }
                }
            }
            if (!full) {
#pragma unroll
                for (int nb = 0; nb < QB; ++nb)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int li = __shfl_sync(0xffffffffu, lane_lim, nb * 8 + 2 * quad + c);
                        const int lo = p.window > 0 ? li - p.window : -1;
#pragma unroll
                        for (int i = 0; i < 2 * KB; ++i) {
                            const int key = key0 + kg + 8 * i;
                            bool see = key <= li && key > lo;
                            if (TREE && see && key >= prior) see = (p.anc[b * p.T + (li - prior)] >> (key - prior)) & 1ull;
                            if (!see) sc[i >> 1][nb][2 * (i & 1) + c] = -INFINITY;
                        }
                    }
            }
            float over = -INFINITY;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int nb = 0; nb < QB; ++nb)
#pragma unroll
                    for (int e = 0; e < 4; ++e) over = fmaxf(over, sc[kb][nb][e]);
            if (__any_sync(0xffffffffu, fresh || over > kLazyRescale || ve > vexp)) {
                // Move the references; O, l, the zero points' sum and the scores follow.
                ve = max(vexp, __reduce_max_sync(0xffffffffu, ve));
                const float fv =
                    __uint_as_float(static_cast<uint32_t>(max(0, 127 + static_cast<int>(vexp) - static_cast<int>(ve))) << 23);
                vexp = ve;
                vmul = __uint_as_float((260u - vexp) << 23);
                fresh = false;
#pragma unroll
                for (int nb = 0; nb < QB; ++nb) {
                    float f[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float t = -INFINITY;
#pragma unroll
                        for (int kb = 0; kb < KB; ++kb) t = fmaxf(t, fmaxf(sc[kb][nb][c], sc[kb][nb][2 + c]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
                        // (t is relative to the old reference, which is 0 before a row's first key)
                        const bool mv = t > kLazyRescale || (m[nb][c] == -INFINITY && t != -INFINITY);
                        const float by = mv ? t : 0.f;
                        f[c] = !mv ? 1.f : m[nb][c] == -INFINITY ? 0.f : ptx::ex2(-t);
                        if (mv) {
                            m[nb][c] = t - nm[nb][c];
                            nm[nb][c] = -m[nb][c];
                        }
                        fresh |= m[nb][c] == -INFINITY;
#pragma unroll
                        for (int kb = 0; kb < KB; ++kb) {
                            sc[kb][nb][c] -= by;
                            sc[kb][nb][2 + c] -= by;
                        }
                        l[nb][c] *= f[c];
                        f[c] *= fv;
                        zs[nb][c] *= f[c];
                        zs[nb][2 + c] *= f[c];
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
                // Weights: p into l, p s_v (f16) into the products.
                const float vs0 = q4::step_of(vw[kb][0]) * vmul, vs1 = q4::step_of(vw[kb][1]) * vmul;
                uint32_t pb[QB][2];
#pragma unroll
                for (int nb = 0; nb < QB; ++nb) {
                    float pw[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float pe = ptx::ex2(sc[kb][nb][e]);
                        l[nb][e & 1] += pe;
                        pw[e] = pe * ((e < 2) ? vs0 : vs1);
                    }
                    if (!full) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (sc[kb][nb][e] == -INFINITY) pw[e] = 0.f;  // (a NaN step that this query does not see)
                    }
                    const uint32_t h0 = ptx::pack_f16x2(pw[0], pw[1]), h1 = ptx::pack_f16x2(pw[2], pw[3]);
                    pb[nb][0] = transpose8x8(h0);
                    pb[nb][1] = transpose8x8(h1);
                }
                // O^T += V^T P^T, and the zero points'.
                {
                    // (Accumulator row g's key has its zero point here; the transpose
                    // gives each thread those of its k index's keys.)
                    const uint32_t z0 = transpose8x8(zero_pair(vw[kb][0], vw[kb][0])), z8 = transpose8x8(zero_pair(vw[kb][1], vw[kb][1]));
                    const uint32_t a[4] = {z0, z0, z8, z8};
#pragma unroll
                    for (int nb = 0; nb < QB; ++nb) ptx::mma_f16_16816(zs[nb], a, pb[nb][0], pb[nb][1]);
                }
                uint32_t va0[VW], vb0[VW], va8[VW], vb8[VW];
                const uint32_t pa = sV + vpiece_a + (at + kb * 16) * S::kRowB, pc = sV + vpiece_b + (at + kb * 16) * S::kRowB;
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

        for (; mine < it_end; mine += party.step()) {
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

            if (p.append_new && key0 + kWarpKeys > prior)
                append_slice<D>(p, b, kvh, prior, nn, key0, koff, lane, smem + stage * S::kStageB);

            if (key0 + kWarpKeys - 1 <= min_lim && key0 > max_lo && (!TREE || key0 + kWarpKeys <= prior)) {
#pragma unroll 1
                for (int k = 0; k < kWarpKeys; k += KB * 16) attend(std::true_type(), key0 + k, koff + k, sK, sV, sS);
            } else {
#pragma unroll 1
                for (int k = 0; k < kWarpKeys; k += KB * 16)
                    if (key0 + k < extent && key0 + k + KB * 16 - 1 > min_lo) attend(std::false_type(), key0 + k, koff + k, sK, sV, sS);
            }
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
                            e[v] = (o[nb][4 * i + c][h] - zs[nb][h]) * 262144.f * real;  // 2^24 2^-6
                            e[v + 2] = fmaf(o[nb][4 * i + c][2 + h], 0.0625f, -zs[nb][h]) * 262144.f * real;
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
            party.sync();
            // Merge the party's in the order of the warps, and write the unit's output
            // (it saw all of it) or the part's partial.
            const size_t out_row0 = seg->row0;
            const uint32_t out_valid = seg->valid;
            const int unit = seg->unit;
            const bool sole = nseg == cur.nt;
            constexpr int C4 = D / 4;
            const int rank = party.rank(tid), w0 = party.lead() * kTileWarps, w1 = party.end() * kTileWarps;
            for (int idx = rank; idx < S::kRows * C4; idx += party.threads()) {
                const int lr = idx / C4, c4 = idx - lr * C4;
                if (!((out_valid >> lr) & 1u)) continue;
                const float* st = obuf + lr * PS;
                float M = -INFINITY;
#pragma unroll 4
                for (int w = w0; w < w1; ++w) M = fmaxf(M, st[w * S::kRows * PS + D]);
                const float Mu = M == -INFINITY ? 0.f : M;
                float L = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int w = w0; w < w1; ++w) {
                    const float* sw = st + w * S::kRows * PS;
                    const float f = ptx::ex2(sw[D] - Mu);
                    const float4 v = reinterpret_cast<const float4*>(sw)[c4];
                    L = fmaf(sw[D + 1], f, L);
                    acc.x = fmaf(v.x, f, acc.x);
                    acc.y = fmaf(v.y, f, acc.y);
                    acc.z = fmaf(v.z, f, acc.z);
                    acc.w = fmaf(v.w, f, acc.w);
                }
                write_row<D>(p, out_row0 + lr, c4, acc, M, L, sole, unit + party.part(), lr);
            }
            if (!sole && p.counters)
                finish_unit<D, S::kRows>(p, unit, seg->unit_tile, cur.nt, wp.total_tiles(), shares(wp), out_row0, out_valid, party, rank, segs[party.lead()].flag);
            party.sync();
        }
        x += nseg;
        cur.j = cur.nt - 1;  // (the next unit; past the last one nothing reads it)
        if (x < x1) cur.advance(wp);
    }
}

template <int D, int QB, bool DP, bool TREE, bool SPLIT>
cudaError_t launch_q4_t(const DecodeParams& p, int grid, cudaStream_t stream) {
    using S = Q4Shape<D, QB>;
    static bool attr_set = false;
    if (!attr_set) {
        cudaError_t e = cudaFuncSetAttribute(decode_q4_kernel<D, QB, DP, TREE, SPLIT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
        if (e != cudaSuccess) return e;
        attr_set = true;
    }
    cudaError_t e = launch_pdl(decode_q4_kernel<D, QB, DP, TREE, SPLIT>, dim3(grid), dim3(S::kThreads), S::kSmem, stream, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <int D, int QB>
cudaError_t launch_q4_shape(const DecodeParams& p, int grid, cudaStream_t stream) {
    const bool split = p.num_ctas > grid;  // (never with a draft tree)
    if (p.anc) return p.dplan || split ? cudaErrorInvalidValue : launch_q4_t<D, QB, false, true, false>(p, grid, stream);
    if (split) return p.dplan ? launch_q4_t<D, QB, true, false, true>(p, grid, stream) : launch_q4_t<D, QB, false, false, true>(p, grid, stream);
    return p.dplan ? launch_q4_t<D, QB, true, false, false>(p, grid, stream) : launch_q4_t<D, QB, false, false, false>(p, grid, stream);
}

}  // namespace

cudaError_t launch_decode_q4(const DecodeParams& p, int grid, int d, cudaStream_t stream) {
    if (d == 128) return p.RPB == 8 ? launch_q4_shape<128, 1>(p, grid, stream) : launch_decode_q4_wide(p, grid, stream);
    if (d != 64) return cudaErrorInvalidValue;
    switch (p.RPB) {
        case 8: return launch_q4_shape<64, 1>(p, grid, stream);
        case 16: return launch_q4_shape<64, 2>(p, grid, stream);
        case 24: return launch_q4_shape<64, 3>(p, grid, stream);
        case 32: return launch_q4_shape<64, 4>(p, grid, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace kvc
