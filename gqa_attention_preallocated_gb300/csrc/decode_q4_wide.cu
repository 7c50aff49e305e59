// Split-KV GQA attention over a 4-bit cache for 9 to 32 query rows per KV head
// at head width 128 (verify, large groups; more rows in blocks of 32).  The
// mathematics, the operand layouts and the ring of stages are those of
// decode_q4.cu; what differs is who holds the output.
//
// There a warp keeps O^T (128 dims) of its own keys, which for 32 query rows
// would be 128 registers a thread.  Here the four warps of a tile exchange
// their weights through shared memory:
//  * Scores: warp w takes keys 32w .. 32w + 31 for all query rows, and writes
//    the weights p s_v (f16) of its keys.
//  * Output: warp (kh, dh) takes keys 64 kh .. + 63 and dims 64 dh .. + 63 for
//    all query rows, 16 registers a block of 8 rows.
// So K and V are unpacked once a tile for up to 32 rows.  The softmax reference
// and V's step exponent are the four warps' in common.  Weights are written on
// the assumption that they stand; the barrier between scores and output, one a
// tile, also ORs the warps' findings that they do not, and then the four redo
// the tile's scores with references moved together (the first tile of a unit,
// and rarely after it: a maximum has to pass the reference by 2^8).  For that
// the sums l are set aside in shared memory before each tile.  The weights'
// buffer is double, so that the next tile's may be written while a slower warp
// still reads.  Two or three such groups take tiles in turn (or have shares of
// their own) and hide each other's barriers.
// The queries' fragments live in shared memory: they would be 16 registers a
// block of 8 rows.
//
// Measured, 64 rows of 4096 tokens, 8 KV heads (287 MB): 16 query rows 107 us, 24
// rows 133, 32 rows 174 (the tensor-core kernel: 218).  Bound by issue and its
// waits, not by a pipe: of the cycles 40 % issue, 35 % have the tensor pipe busy.
// So warps count: the copying warps give up registers, and 24 rows ran 151 us with
// two groups of 232 registers, 138 with three of 160; 32 rows 182 with three
// (spills), 177 with two; scoring 32 keys side by side took 112 us where 16 at a
// time took 122 (16 rows).  Running a tile's output beside the next one's scores
// in the same warp gained nothing (162 us against 151): the other groups fill
// those cycles already.

#include "q4_splitkv.cuh"

namespace kvc {

namespace {

using namespace q4;

// QB: blocks of 8 query rows.
template <int QB>
struct WideShape {
    static constexpr int D = 128;
    // Groups of four warps: as many as leave a thread the registers it needs.
    static constexpr int kGroups = q4_groups(D, 8 * QB);
    static constexpr int kCW = kGroups * kTileWarps;
    static constexpr int kCT = kCW * 32;
    static constexpr int kThreads = kCT + 128;        // a warpgroup copies (a warp a group of the others)
    // Registers of a thread at launch, and of a computing and a copying one after
    // the split: 384 x 160 + 128 x 32 = 512 x 128, or 256 x 232 + 128 x 40 = 384 x 168.
    static constexpr int kLaunchRegs = kGroups == 3 ? 128 : 168;
    static constexpr int kRegs = kGroups == 3 ? 160 : 232, kCopyRegs = kGroups == 3 ? 32 : 40;
    static_assert(kCT * kRegs + 128 * kCopyRegs <= kThreads * kLaunchRegs && kThreads * kLaunchRegs <= 65536, "register split");
    static constexpr int kRows = 8 * QB;
    static constexpr int kStageB = Stage<D>::kBytes, kRowB = Stage<D>::kRowB, kCodeB = Stage<D>::kCodeB;
    static constexpr int kPS = D + 4;                 // floats of a partial's row: O, m, l, pad
    static constexpr int kPRow = kKT * 2 + 16;        // bytes of a weight row (the pad spreads 8 rows over all banks)
    // Behind the stages: for each group the weights of two tiles [2][row] and the
    // sums l set aside [block][thread], at a segment's end its state [row][kPS];
    // query fragments [group][QB][4 words][32 lanes] of 16 bytes, (sum of q, score
    // factor) [group][row], each warp's maxima [group][warp][row] and exponents,
    // sums l and the zero points' [group][warp][row], references [group][row].
    static constexpr int kPhalf = kRows * kPRow;      // one tile's weights of a group
    static constexpr int kTile = 2 * kPhalf + QB * 128 * 8, kState = kRows * kPS * 4;
    static constexpr int kGroupB = kTile > kState ? kTile : kState;
    static constexpr int kQbuf = QB * 4 * 32 * 16;
    static constexpr int kOffQ = kGroups * kGroupB, kOffQs = kOffQ + kGroups * kQbuf, kOffMx = kOffQs + kGroups * kRows * 8,
                         kOffVe = kOffMx + kCW * kRows * 4, kOffLz = kOffVe + 64, kOffM = kOffLz + kCW * kRows * 8,
                         kMisc = kOffM + kGroups * kRows * 4;
    static constexpr int kFit = (232448 - 1024 - 512 - kMisc) / kStageB;
    static constexpr int kStages = kFit / kGroups * kGroups;
    static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStageB + kMisc + 2 * kStages * 8 + 16 + kGroups * sizeof(Segment);
    static_assert(kStages >= 2 * kGroups, "a stage to read and one to fill for every group");
    static_assert(kSmem <= 232448 && kMisc % 16 == 0 && kGroupB % 16 == 0 && kOffLz % 8 == 0, "shared memory map");
};

// Barrier of a group's 128 threads that also ORs one bit.
__device__ __forceinline__ bool barrier_or(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\tbarrier.cta.red.or.pred b, %2, 128, a;\n\t"
        "selp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(v)), "r"(id)
        : "memory");
    return r != 0;
}

template <int QB, bool DP, bool TREE, bool SPLIT>
__global__ void __launch_bounds__(WideShape<QB>::kThreads, 1)
    decode_q4_wide_kernel(const __grid_constant__ DecodeParams p) {
    using S = WideShape<QB>;
    constexpr int D = S::D, kStages = S::kStages, PS = S::kPS;
    constexpr int kChunks = kWarpKeys / 16;  // blocks of 16 keys, scored side by side

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* misc = smem + static_cast<size_t>(kStages) * S::kStageB;
    uint64_t* bars = reinterpret_cast<uint64_t*>(misc + S::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * kStages);
    volatile Segment* segs = reinterpret_cast<volatile Segment*>(bars + 2 * kStages + 2);  // a group's

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Part<DP> wp{p};

    const uint32_t stage0 = ptx::smem_addr(smem), misc0 = ptx::smem_addr(misc);
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

    if (warp >= S::kCW) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kCopyRegs));
        if (grp < S::kGroups && x0 < x1)
            produce<D, kStages, DP>(p, wp, x0, x1, party, lane, stage0, bar0, abort_flag);
        return;
    }

    // ------------------------------------------------------------------ consumers
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegs));
    if (x0 >= x1) return;
    const int gw = warp % kTileWarps;
    const int kh = gw >> 1, dh = gw & 1;  // output: this warp's half of the keys and of the dims
    const int koff = gw * kWarpKeys;      // scores: its keys of a tile
    const int quad = lane & 3, g = lane >> 2;
    const int kg = perm8<D>(g), va = perm8<D>(2 * quad), vb = perm8<D>(2 * quad + 1);
    const uint32_t kpiece = kg * S::kRowB + quad * 16;
    const uint32_t vpiece_a = (kh * 64 + va) * S::kRowB + dh * 32 + g * 4;
    const uint32_t vpiece_b = (kh * 64 + vb) * S::kRowB + dh * 32 + g * 4;
    const uint32_t pbuf = misc0 + grp * S::kGroupB;
    const uint32_t pstore = pbuf + g * S::kPRow + (2 * quad) * 2;  // + half, + block of rows, + key
    const uint32_t pload = pbuf + (lane & 7) * S::kPRow + (kh * 64 + (lane >> 3) * 8) * 2;
    float2* qsum = reinterpret_cast<float2*>(misc + S::kOffQs) + grp * S::kRows;
    float* mxbuf = reinterpret_cast<float*>(misc + S::kOffMx) + grp * kTileWarps * S::kRows;
    uint32_t* vebuf = reinterpret_cast<uint32_t*>(misc + S::kOffVe) + grp * kTileWarps;
    float2* lzbuf = reinterpret_cast<float2*>(misc + S::kOffLz);
    float* mbuf = reinterpret_cast<float*>(misc + S::kOffM);
    float2* save = reinterpret_cast<float2*>(misc + grp * S::kGroupB + 2 * S::kPhalf) + (tid & 127);
    const uint32_t qfrag = misc0 + S::kOffQ + grp * S::kQbuf + lane * 16;
    volatile Segment* seg = segs + grp;

    Cursor<DP, kKT> cur;
    cur.init(wp, x0);
    int mine = party.first_tile(), stage = grp, phase = 0;

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
        const int seg_tile0 = (cur.t0 + j0) * kKT - (x - x0) * kKT;    // + it * kKT: the tile's first key
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

        // Query fragments (as in decode_q4.cu): warp nb writes block nb's, and its
        // rows' sums and score factors.
        {
            if (gw < QB) {
                const uint4* qrow = nullptr;
                if ((valid >> (gw * 8 + g)) & 1u)
                    qrow = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (row0 + gw * 8 + g) * D + quad * 32);
                uint4 w[4];
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] = qrow ? __ldg(qrow + i) : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) top = max(top, max(u[c] & 0x7FFFu, (u[c] >> 16) & 0x7FFFu));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = max(14, static_cast<int>(top >> 7));
                const float f = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);  // 2^(141 - e)
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                    uint32_t h[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float a0 = __uint_as_float(u[c] << 16) * f, a1 = __uint_as_float(u[c] & 0xFFFF0000u) * f;
                        sum += a0 + a1;
                        const float t = (c & 1) ? 0.0625f : 1.f;
                        h[c] = ptx::pack_f16x2(a0 * t, a1 * t);
                    }
                    *reinterpret_cast<uint4*>(misc + S::kOffQ + grp * S::kQbuf + ((gw * 4 + i) * 32 + lane) * 16) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (quad == 0)  // 2^-24 sum, and 2^(e - 141) 2^24 log2(e) / sqrt(d)
                    qsum[gw * 8 + g] = make_float2(sum * 5.9604644775390625e-8f,
                                                     p.scale_log2 * __uint_as_float(static_cast<uint32_t>(min(254, e + 10)) << 23));
            }
            ptx::named_barrier_sync(2 + grp, 128);
        }

        // The segment's state: O^T of this warp's keys and dims; the negative of
        // the group's references (0 before a row's first key; `seen` has a bit for
        // each row that has one, or is no query); sums over this warp's scored keys.
        float o[QB][4][4];
        float nm[QB][2], l[QB][2], zs[QB][4];
        uint32_t seen = 0;
        uint32_t vexp = kMinExp;
        float vmul = __uint_as_float((260u - kMinExp) << 23);  // 2^(133 - vexp)
#pragma unroll
        for (int nb = 0; nb < QB; ++nb) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (!((valid >> (nb * 8 + 2 * quad + c)) & 1u)) seen |= 1u << (2 * nb + c);
                nm[nb][c] = l[nb][c] = zs[nb][c] = zs[nb][2 + c] = 0.f;
            }
#pragma unroll
            for (int mb = 0; mb < 4; ++mb) o[nb][mb][0] = o[nb][mb][1] = o[nb][mb][2] = o[nb][mb][3] = 0.f;
        }
        constexpr uint32_t kAll = (1u << (2 * QB)) - 1;

        // From raw scores to weights, for 16 keys from key0 on: the weights written
        // at `pst`, the rows' maxima, relative to the references, into mx, V's
        // largest exponent into ve.  full: every valid query of the block sees every
        // key.
        float mx[QB][2];
        uint32_t ve;
        auto settle = [&](const bool full, const int key0, uint32_t (&kw)[2], uint32_t (&vw)[2], float (&sc)[QB][4], const uint32_t pst) {
            if (!full) {
                // (Keys that no query of the block sees: no step, so that neither a
                // stale word nor its exponent enters.)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int key = key0 + kg + 8 * h;
                    if (key >= extent || key <= min_lo) kw[h] = vw[h] = 0u;
                }
            }
            const float ks0 = step_of(kw[0]), ks1 = step_of(kw[1]);
            const float kz0 = -zero_f32(kw[0]), kz1 = -zero_f32(kw[1]);
#pragma unroll
            for (int nb = 0; nb < QB; ++nb) {
                const float4 qs = *reinterpret_cast<const float4*>(qsum + nb * 8 + 2 * quad);  // of two rows
                sc[nb][0] = fmaf(fmaf(kz0, qs.x, sc[nb][0]), ks0 * qs.y, nm[nb][0]);
                sc[nb][1] = fmaf(fmaf(kz0, qs.z, sc[nb][1]), ks0 * qs.w, nm[nb][1]);
                sc[nb][2] = fmaf(fmaf(kz1, qs.x, sc[nb][2]), ks1 * qs.y, nm[nb][0]);
                sc[nb][3] = fmaf(fmaf(kz1, qs.z, sc[nb][3]), ks1 * qs.w, nm[nb][1]);
            }
            if (!full) {
#pragma unroll
                for (int nb = 0; nb < QB; ++nb)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int li = __shfl_sync(0xffffffffu, lane_lim, nb * 8 + 2 * quad + c);
                        const int lo = p.window > 0 ? li - p.window : -1;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int key = key0 + kg + 8 * h;
                            bool see = key <= li && key > lo;
                            if (TREE && see && key >= prior) see = (p.anc[b * p.T + (li - prior)] >> (key - prior)) & 1ull;
                            if (!see) sc[nb][2 * h + c] = -INFINITY;
                        }
                    }
            }
            // (a NaN step has no exponent: it stays NaN under any factor)
            ve = max(ve, max((vw[0] >> 23) == 255u ? 0u : vw[0] >> 23, (vw[1] >> 23) == 255u ? 0u : vw[1] >> 23));
            const float vs0 = step_of(vw[0]) * vmul, vs1 = step_of(vw[1]) * vmul;
#pragma unroll
            for (int nb = 0; nb < QB; ++nb) {
                float pw[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    mx[nb][e & 1] = fmaxf(mx[nb][e & 1], sc[nb][e]);
                    const float pe = ptx::ex2(sc[nb][e]);
                    l[nb][e & 1] += pe;
                    pw[e] = pe * ((e < 2) ? vs0 : vs1);
                }
                if (!full) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (sc[nb][e] == -INFINITY) pw[e] = 0.f;  // (a NaN step that this query does not see)
                }
                const uint32_t h0 = ptx::pack_f16x2(pw[0], pw[1]), h1 = ptx::pack_f16x2(pw[2], pw[3]);
                const uint32_t to = pst + nb * 8 * S::kPRow;
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(transpose8x8(h0)) : "memory");
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + 16), "r"(transpose8x8(h1)) : "memory");
            }
        };
        // The same for 16 kChunks keys from key0 (row `at` of the tile) on.
        auto weigh = [&](const bool full, const int key0, const int at, const uint32_t sK, const uint32_t sS, const uint32_t pst) {
            // S^T of all its keys first: 2 QB chains of products side by side, and a
            // query fragment read once for them.
            float sa[kChunks][QB][4];
            uint32_t kwa[kChunks][2], vwa[kChunks][2], kc[kChunks][2][4];
#pragma unroll
            for (int u = 0; u < kChunks; ++u) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    kwa[u][h] = lds32(sS + (at + 16 * u + kg + 8 * h) * 4);
                    vwa[u][h] = lds32(sS + (kKT + at + 16 * u + kg + 8 * h) * 4);
                    const uint4 c = ptx::ld_shared_v4(sK + kpiece + (at + 16 * u + 8 * h) * S::kRowB);
                    kc[u][h][0] = c.x, kc[u][h][1] = c.y, kc[u][h][2] = c.z, kc[u][h][3] = c.w;
                }
#pragma unroll
                for (int nb = 0; nb < QB; ++nb) sa[u][nb][0] = sa[u][nb][1] = sa[u][nb][2] = sa[u][nb][3] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t a[kChunks][4], c[kChunks][4];
#pragma unroll
                for (int u = 0; u < kChunks; ++u) {
                    const uint32_t x0w = kc[u][0][i], x1w = kc[u][1][i], y0w = x0w >> 8, y1w = x1w >> 8;
                    a[u][0] = x0w & 0x000F000Fu, a[u][1] = x1w & 0x000F000Fu, a[u][2] = x0w & 0x00F000F0u, a[u][3] = x1w & 0x00F000F0u;
                    c[u][0] = y0w & 0x000F000Fu, c[u][1] = y1w & 0x000F000Fu, c[u][2] = y0w & 0x00F000F0u, c[u][3] = y1w & 0x00F000F0u;
                }
#pragma unroll
                for (int nb = 0; nb < QB; ++nb) {
                    const uint4 f = ptx::ld_shared_v4(qfrag + (nb * 4 + i) * 512);
#pragma unroll
                    for (int u = 0; u < kChunks; ++u) ptx::mma_f16_16816(sa[u][nb], a[u], f.x, f.y);
#pragma unroll
                    for (int u = 0; u < kChunks; ++u) ptx::mma_f16_16816(sa[u][nb], c[u], f.z, f.w);
                }
            }
#pragma unroll
            for (int u = 0; u < kChunks; ++u) settle(full, key0 + 16 * u, kwa[u], vwa[u], sa[u], pst + u * 32);
        };

        for (uint32_t half = 0; mine < it_end; mine += party.step(), half ^= S::kPhalf) {
            // (On expiry as in decode_q4.cu: record it and carry on.)
            if (!ptx::mbar_try_wait(bar0 + 8 * stage, phase) &&
                !ptx::mbar_wait_bounded(bar0 + 8 * stage, phase, *abort_flag ? 0ull : kWaitLimitNs)) {
                atomicExch(p.err, kDevTimeoutFull);
                *abort_flag = 1;
            }
            const uint32_t sK = stage0 + stage * S::kStageB, sV = sK + S::kCodeB, sS = sV + S::kCodeB;
            const int tile0 = seg_tile0 + mine * kKT, key0 = tile0 + koff;
            if (p.append_new && key0 + kWarpKeys > prior)
                append_slice<D>(p, b, kvh, prior, nn, key0, koff, lane, smem + stage * S::kStageB);

            bool moved = false;
#pragma unroll
            for (int nb = 0; nb < QB; ++nb) save[nb * 128] = make_float2(l[nb][0], l[nb][1]);
            const uint32_t pst = pstore + half + koff * 2;
            const bool full = key0 + kWarpKeys - 1 <= min_lim && key0 > max_lo && (!TREE || key0 + kWarpKeys <= prior);
            // Once, and again with moved references where they do not stand (one
            // copy of the code: its second and third were slower to fetch than to
            // run).
            for (;;) {
                ve = 0;
#pragma unroll
                for (int nb = 0; nb < QB; ++nb) mx[nb][0] = mx[nb][1] = -INFINITY;
                weigh(full, key0, koff, sK, sS, pst);
                bool move = seen != kAll || ve > vexp;
#pragma unroll
                for (int nb = 0; nb < QB; ++nb) move |= fmaxf(mx[nb][0], mx[nb][1]) > kLazyRescale;
                if (!barrier_or(2 + grp, move && !moved)) break;
                moved = true;
                // The group's rows' maxima; then the references, O and the sums (as
                // they were before the tile) move.
                ve = __reduce_max_sync(0xffffffffu, ve);
#pragma unroll
                for (int nb = 0; nb < QB; ++nb) {
                    const float2 v = save[nb * 128];
                    l[nb][0] = v.x, l[nb][1] = v.y;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) mx[nb][c] = fmaxf(mx[nb][c], __shfl_xor_sync(0xffffffffu, mx[nb][c], d));
                        if (g == 0) mxbuf[gw * S::kRows + nb * 8 + 2 * quad + c] = mx[nb][c];
                    }
                }
                if (lane == 0) vebuf[gw] = ve;
                ptx::named_barrier_sync(2 + grp, 128);
                ve = max(max(vexp, max(vebuf[0], vebuf[1])), max(vebuf[2], vebuf[3]));
                const float fv =
                    __uint_as_float(static_cast<uint32_t>(max(0, 127 + static_cast<int>(vexp) - static_cast<int>(ve))) << 23);
                vexp = ve;
                vmul = __uint_as_float((260u - vexp) << 23);
#pragma unroll
                for (int nb = 0; nb < QB; ++nb) {
                    float f[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int r = nb * 8 + 2 * quad + c;
                        const uint32_t bit = 1u << (2 * nb + c);
                        const float t = fmaxf(fmaxf(mxbuf[r], mxbuf[S::kRows + r]),
                                              fmaxf(mxbuf[2 * S::kRows + r], mxbuf[3 * S::kRows + r]));
                        // (t is relative to the old reference, which is 0 before a row's first key)
                        const bool mv = t > kLazyRescale || (!(seen & bit) && t != -INFINITY);
                        f[c] = !mv ? 1.f : !(seen & bit) ? 0.f : ptx::ex2(-t);
                        if (mv) {
                            nm[nb][c] -= t;
                            seen |= bit;
                        }
                        l[nb][c] *= f[c];
                        f[c] *= fv;
                        zs[nb][c] *= f[c];
                        zs[nb][2 + c] *= f[c];
                    }
#pragma unroll
                    for (int mb = 0; mb < 4; ++mb) {
                        o[nb][mb][0] *= f[0];
                        o[nb][mb][1] *= f[1];
                        o[nb][mb][2] *= f[0];
                        o[nb][mb][3] *= f[1];
                    }
                }
            }

            // O^T += V^T P^T, 32 keys at a time, up to the last visible one.
#pragma unroll
            for (int kp = 0; kp < 2; ++kp) {
                if (tile0 + kh * 64 + kp * 32 >= extent) break;
                uint32_t pb[QB][4];
#pragma unroll
                for (int nb = 0; nb < QB; ++nb)
                    ptx::ldmatrix_x4(pload + half + nb * 8 * S::kPRow + kp * 64, pb[nb][0], pb[nb][1], pb[nb][2], pb[nb][3]);
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    if (dh == 0) {  // the zero points' sum (16 equal rows)
                        const uint32_t zw = sS + (kKT + kh * 64 + kp * 32 + kb * 16) * 4;
                        const uint32_t z0 = zero_pair(lds32(zw + va * 4), lds32(zw + vb * 4));
                        const uint32_t z8 = zero_pair(lds32(zw + va * 4 + 32), lds32(zw + vb * 4 + 32));
                        const uint32_t a[4] = {z0, z0, z8, z8};
#pragma unroll
                        for (int nb = 0; nb < QB; ++nb) ptx::mma_f16_16816(zs[nb], a, pb[nb][2 * kb], pb[nb][2 * kb + 1]);
                    }
                    const uint32_t pa = sV + vpiece_a + (kp * 32 + kb * 16) * S::kRowB, pc = sV + vpiece_b + (kp * 32 + kb * 16) * S::kRowB;
                    const uint32_t a0 = lds32(pa), b0 = lds32(pc), a8 = lds32(pa + 8 * S::kRowB), b8 = lds32(pc + 8 * S::kRowB);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // even, then odd values of the word
                        const uint32_t sel = h ? 0x7632u : 0x5410u;
                        const uint32_t u = ptx::prmt(a0, b0, sel), v = ptx::prmt(a8, b8, sel);
                        const uint32_t u8 = u >> 8, v8 = v >> 8;
                        const uint32_t a[4] = {u & 0x000F000Fu, u & 0x00F000F0u, v & 0x000F000Fu, v & 0x00F000F0u};
                        const uint32_t c[4] = {u8 & 0x000F000Fu, u8 & 0x00F000F0u, v8 & 0x000F000Fu, v8 & 0x00F000F0u};
#pragma unroll
                        for (int nb = 0; nb < QB; ++nb) {
                            ptx::mma_f16_16816(o[nb][2 * h], a, pb[nb][2 * kb], pb[nb][2 * kb + 1]);
                            ptx::mma_f16_16816(o[nb][2 * h + 1], c, pb[nb][2 * kb], pb[nb][2 * kb + 1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar0 + 8 * (kStages + stage));
            stage += S::kGroups;
            if (stage >= kStages) {
                stage -= kStages;
                phase ^= 1;
            }
        }

        // The segment's end: the group's state into shared memory (over its weights,
        // once no warp reads them) in real units.
        ptx::named_barrier_sync(2 + grp, 128);
        const float real = 0.015625f * __uint_as_float(vexp << 23);  // 2^(vexp - 133), as a product that stays normal
        // (Keys' second halves are added to the first.)
        if (kh == 1) ptx::named_barrier_sync(2 + grp, 128);
#pragma unroll
        for (int nb = 0; nb < QB; ++nb)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    l[nb][c] += __shfl_xor_sync(0xffffffffu, l[nb][c], d);
                }
                const int lr = nb * 8 + 2 * quad + c;
                float e[8];  // dims 0 .. 7: blocks 0 .. 3 hold (0, 2), (4, 6), (1, 3), (5, 7)
#pragma unroll
                for (int mb = 0; mb < 4; ++mb) {
                    const int v = (mb & 1) * 4 + (mb >> 1);
                    e[v] = o[nb][mb][c] * 16777216.f * real;
                    e[v + 2] = o[nb][mb][2 + c] * 1048576.f * real;
                }
                float4* d4 = reinterpret_cast<float4*>(misc + grp * S::kGroupB) + lr * (PS / 4) + dh * 16 + g * 2;
                if (kh == 1) {
                    const float4 u = d4[0], v = d4[1];
                    e[0] += u.x, e[1] += u.y, e[2] += u.z, e[3] += u.w;
                    e[4] += v.x, e[5] += v.y, e[6] += v.z, e[7] += v.w;
                }
                d4[0] = make_float4(e[0], e[1], e[2], e[3]);
                d4[1] = make_float4(e[4], e[5], e[6], e[7]);
                if (g == 0) {
                    lzbuf[warp * S::kRows + lr] = make_float2(l[nb][c], zs[nb][c] * 16777216.f * real);  // (0 with dh = 1)
                    if (gw == 0) mbuf[grp * S::kRows + lr] = (seen >> (2 * nb + c)) & 1u ? -nm[nb][c] : -INFINITY;
                }
            }
        if (kh == 0) ptx::named_barrier_sync(2 + grp, 128);
        party.sync();
        // Merge the party's groups in their order, and write the unit's output (it
        // saw all of it) or the part's partial.
        const size_t out_row0 = seg->row0;
        const uint32_t out_valid = seg->valid;
        const int unit = seg->unit;
        const bool sole = nseg == cur.nt;
        constexpr int C4 = D / 4;
        const int rank = party.rank(tid);
        for (int idx = rank; idx < S::kRows * C4; idx += party.threads()) {
            const int lr = idx / C4, c4 = idx - lr * C4;
            if (!((out_valid >> lr) & 1u)) continue;
            // A group's sum, zero points' sum and reference.
            auto sums = [&](int i, float& gl, float& gz) {
                gl = gz = 0.f;
#pragma unroll
                for (int w = 0; w < kTileWarps; ++w) {
                    const float2 lz = lzbuf[(i * kTileWarps + w) * S::kRows + lr];
                    gl += lz.x;
                    gz += lz.y;
                }
                const float m = mbuf[i * S::kRows + lr];
                return m == -INFINITY && gl != 0.f ? 0.f : m;  // (a row whose every score is NaN keeps that)
            };
            float M = -INFINITY, gl, gz;
            for (int i = party.lead(); i < party.end(); ++i) M = fmaxf(M, sums(i, gl, gz));
            const float Mu = M == -INFINITY ? 0.f : M;
            float L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i = party.lead(); i < party.end(); ++i) {
                const float f = ptx::ex2(sums(i, gl, gz) - Mu);
                const float4 u = reinterpret_cast<const float4*>(misc + i * S::kGroupB)[lr * (PS / 4) + c4];
                L = fmaf(gl, f, L);
                acc.x = fmaf(u.x - gz, f, acc.x);
                acc.y = fmaf(u.y - gz, f, acc.y);
                acc.z = fmaf(u.z - gz, f, acc.z);
                acc.w = fmaf(u.w - gz, f, acc.w);
            }
            write_row<D>(p, out_row0 + lr, c4, acc, M, L, sole, unit + party.part(), lr);
        }
        if (!sole && p.counters)
            finish_unit<D, S::kRows>(p, unit, seg->unit_tile, cur.nt, wp.total_tiles(), shares(wp), out_row0, out_valid, party, rank, segs[party.lead()].flag);
        party.sync();
        x += nseg;
        cur.j = cur.nt - 1;  // (the next unit; past the last one nothing reads it)
        if (x < x1) cur.advance(wp);
    }
}

template <int QB, bool DP, bool TREE, bool SPLIT>
cudaError_t launch_wide_t(const DecodeParams& p, int grid, cudaStream_t stream) {
    using S = WideShape<QB>;
    static bool attr_set = false;
    if (!attr_set) {
        cudaError_t e = cudaFuncSetAttribute(decode_q4_wide_kernel<QB, DP, TREE, SPLIT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
        if (e != cudaSuccess) return e;
        // The registers that the computing warps take must be there at launch: with
        // fewer they would wait for them for ever.
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, decode_q4_wide_kernel<QB, DP, TREE, SPLIT>);
        if (e != cudaSuccess) return e;
        if ((fa.numRegs + 7) / 8 * 8 < S::kLaunchRegs) return cudaErrorInvalidConfiguration;
        attr_set = true;
    }
    cudaError_t e = launch_pdl(decode_q4_wide_kernel<QB, DP, TREE, SPLIT>, dim3(grid), dim3(S::kThreads), S::kSmem, stream, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <int QB>
cudaError_t launch_wide_qb(const DecodeParams& p, int grid, cudaStream_t stream) {
    const bool split = p.num_ctas > grid;  // (never with a draft tree)
    if (p.anc) return p.dplan || split ? cudaErrorInvalidValue : launch_wide_t<QB, false, true, false>(p, grid, stream);
    if (split) return p.dplan ? launch_wide_t<QB, true, false, true>(p, grid, stream) : launch_wide_t<QB, false, false, true>(p, grid, stream);
    return p.dplan ? launch_wide_t<QB, true, false, false>(p, grid, stream) : launch_wide_t<QB, false, false, false>(p, grid, stream);
}

}  // namespace

cudaError_t launch_decode_q4_wide(const DecodeParams& p, int grid, cudaStream_t stream) {
    switch (p.RPB) {
        case 16: return launch_wide_qb<2>(p, grid, stream);
        case 24: return launch_wide_qb<3>(p, grid, stream);
        case 32: return launch_wide_qb<4>(p, grid, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace kvc
