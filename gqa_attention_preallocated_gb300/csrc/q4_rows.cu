// Writing rows into a 4-bit cache, and reading rows back from any cache.
//
// Append.  Each appended row (one token of one KV head, K or V) is quantised on
// its own: lo = min(0, min x), hi = max(0, max x), s = bf16((hi - lo) / 15),
// z = rint(-lo / s), c = clamp(rint(x / s) + z, 0, 15) in the float32
// operations kvc.h spells out, so the codes are the same bits on every path.
// A group of lanes (the power of two that holds d / 8) owns a row: each lane
// takes one 16-byte vector of eight bf16 values, the range is joined by
// shuffles, and each lane writes one 32-bit word of codes.
// Bound by memory: 2 d bytes read and d / 2 + 4 written a row.
//
// Read back.  A thread writes one 16-byte vector of the result: eight bf16
// values of a 4-bit row (s * (c - z), one rounding), of an FP8 row (code *
// scale, one rounding) or of a bf16 row (a copy), or four fp32 values.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvc_internal.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace kvc {

namespace {

constexpr int kThreads = 256;

// Rows of a thread: with long chunks four, whose loads are in flight together and
// whose divisions are one; with few rows one, for more blocks.  A prompt of 4 x
// 8192 tokens, 8 heads, d = 128: appended in 33 us (46 with one row a
// thread), read back in 26 (37).
constexpr int kManyRows = 4;

// LANES: lanes a row (a power of two, d / 8 or more of them: the others idle).
template <int LANES, int ROWS>
__global__ void __launch_bounds__(kThreads) append_q4_kernel(const __grid_constant__ AppendParams p) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    constexpr int kStep = kThreads / LANES;  // rows a block takes side by side
    const int b = blockIdx.z, h = blockIdx.y >> 1;
    const bool is_v = (blockIdx.y & 1) != 0;
    const int n = p.n_new[b];
    const int sub = threadIdx.x % LANES;
    const int t0 = blockIdx.x * (kStep * ROWS) + threadIdx.x / LANES;
    if (blockIdx.x * (kStep * ROWS) >= n) return;
    const int vecs = p.row_bytes / 16;  // 16-byte vectors of a bf16 row
    const size_t unit = static_cast<size_t>(b) * p.Hkv + h;
    const uint4* src = reinterpret_cast<const uint4*>((is_v ? p.v_new : p.k_new) + unit * p.T * p.row_bytes);
    uint4 val[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int t = t0 + i * kStep;
        val[i] = t < n && sub < vecs ? __ldcs(src + static_cast<size_t>(t) * vecs + sub) : make_uint4(0u, 0u, 0u, 0u);
    }
    uint32_t range[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const uint32_t w[4] = {val[i].x, val[i].y, val[i].z, val[i].w};
        range[i] = q4::range8(w);
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < ROWS; ++i) range[i] = q4::max2(range[i], __shfl_xor_sync(0xffffffffu, range[i], o));
    // The divisions once for all of the group's rows: lane i of every four
    // works out row i, and hands it to the others.
    q4::RowScale mine;
    if constexpr (ROWS == 4) {
        const int i = sub & 3;
        mine = q4::row_scale(i < 2 ? (i == 0 ? range[0] : range[1]) : (i == 2 ? range[2] : range[3]));
    } else {
        static_assert(ROWS == 1, "one row a lane group, or four");
        mine = q4::row_scale(range[0]);
    }
    uint32_t* codes = reinterpret_cast<uint32_t*>(is_v ? p.v_cache : p.k_cache);
    uint32_t* words = is_v ? p.q4.v : p.q4.k;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int t = t0 + i * kStep;
        q4::RowScale rs = mine;
        if constexpr (ROWS == 4) {
            rs.inv = __shfl_sync(0xffffffffu, mine.inv, i, 4);
            rs.word = __shfl_sync(0xffffffffu, mine.word, i, 4);
            rs.plain = rs.inv != 0.f;  // (a step below 2^126 has a reciprocal above 0)
        }
        if (t >= n || sub >= vecs) continue;
        bool bad = false;  // (a position whose block-table entry is bad is not written)
        const int row = phys_row(p.pg, p.ring, p.Hkv, p.max_len, b, h, p.lens[b] + t, &bad);
        if (bad) continue;
        const uint32_t w[4] = {val[i].x, val[i].y, val[i].z, val[i].w};
        codes[static_cast<size_t>(row) * vecs + sub] = q4::encode8(w, rs);
        if (sub == 0) words[q4::scale_index(p.q4, row)] = rs.word;
    }
}

// KIND as in ReadParams; LANES: lanes a row, at least its 16-byte vectors.
template <int KIND, int LANES, int ROWS>
__global__ void __launch_bounds__(kThreads) read_rows_kernel(const __grid_constant__ ReadParams p) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    constexpr int kStep = kThreads / LANES;
    const int b = blockIdx.z, h = blockIdx.y >> 1;
    const bool is_v = (blockIdx.y & 1) != 0;
    const int n = p.count[b];
    const int vecs = p.d * (KIND == kReadF32 ? 4 : 2) / 16;  // 16-byte vectors of a result row
    const int c = threadIdx.x % LANES, t0 = blockIdx.x * (kStep * ROWS) + threadIdx.x / LANES;
    if (t0 >= n || c >= vecs) return;
    const uint8_t* cache = is_v ? p.v_cache : p.k_cache;
    const uint32_t* words = is_v ? p.q4.v : p.q4.k;
    uint4 in[ROWS];       // the vector's stored bytes: 4 (4-bit), 8 (FP8) or 16
    uint32_t sw[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int t = t0 + i * kStep;
        in[i] = make_uint4(0u, 0u, 0u, 0u);
        sw[i] = 0u;
        if (t >= n) continue;
        bool bad = false;  // a bad block-table entry reads as zeros
        const int row = phys_row(p.pg, p.ring, p.Hkv, p.max_len, b, h, p.first[b] + t, &bad);
        if (bad) continue;
        const size_t at = static_cast<size_t>(row) * vecs + c;
        if constexpr (KIND == kReadQ4) {
            in[i].x = __ldg(reinterpret_cast<const uint32_t*>(cache) + at);
            sw[i] = __ldg(words + q4::scale_index(p.q4, row));
        } else if constexpr (KIND == kReadFp8) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(cache) + at);
            in[i].x = w.x, in[i].y = w.y;
        } else {
            in[i] = __ldg(reinterpret_cast<const uint4*>(cache) + at);
        }
    }
    const size_t unit = static_cast<size_t>(b) * p.Hkv + h;
    uint4* dst = reinterpret_cast<uint4*>(is_v ? p.v_out : p.k_out) + unit * p.T * vecs + c;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int t = t0 + i * kStep;
        if (t >= n) continue;
        uint32_t o[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
        if constexpr (KIND == kReadQ4) {
            const uint32_t w = in[i].x;
            const float s = q4::step_of(sw[i]);
            const int z = q4::zero_of(sw[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = ptx::pack_bf16x2(s * static_cast<float>(q4::code_of(w, 2 * e) - z),
                                        s * static_cast<float>(q4::code_of(w, 2 * e + 1) - z));
        } else if constexpr (KIND == kReadFp8) {
            const float s = is_v ? p.vscale[h] : p.kscale[h];
            const uint32_t u[2] = {in[i].x, in[i].y};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t f[2];
                ptx::e4m3x4_to_f16x2x2(u[e], f[0], f[1]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    __half2 hh;
                    memcpy(&hh, &f[j], 4);
                    const float2 v = __half22float2(hh);
                    o[2 * e + j] = ptx::pack_bf16x2(v.x * s, v.y * s);
                }
            }
        }
        __stcs(dst + static_cast<size_t>(t) * vecs, make_uint4(o[0], o[1], o[2], o[3]));
    }
}

template <typename P>
cudaError_t launch_chained(void (*kernel)(P), dim3 grid, cudaStream_t stream, const P& p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

// Grid of a launch over `rows` rows a (K or V, KV head, batch row).
template <int LANES, int ROWS>
dim3 rows_grid(int rows, int Hkv, int B) {
    constexpr int per_block = kThreads / LANES * ROWS;
    return dim3(static_cast<unsigned>((rows + per_block - 1) / per_block), 2u * Hkv, B);
}

template <int LANES>
cudaError_t launch_append_lanes(const AppendParams& p, int rows, cudaStream_t stream) {
    return rows >= kManyRows * (kThreads / LANES)
               ? launch_chained(append_q4_kernel<LANES, kManyRows>, rows_grid<LANES, kManyRows>(rows, p.Hkv, p.B), stream, p)
               : launch_chained(append_q4_kernel<LANES, 1>, rows_grid<LANES, 1>(rows, p.Hkv, p.B), stream, p);
}

template <int KIND, int LANES>
cudaError_t launch_read_lanes(const ReadParams& p, int rows, cudaStream_t stream) {
    return rows >= kManyRows * (kThreads / LANES)
               ? launch_chained(read_rows_kernel<KIND, LANES, kManyRows>, rows_grid<LANES, kManyRows>(rows, p.Hkv, p.B), stream, p)
               : launch_chained(read_rows_kernel<KIND, LANES, 1>, rows_grid<LANES, 1>(rows, p.Hkv, p.B), stream, p);
}

template <int KIND>
cudaError_t launch_read_kind(const ReadParams& p, int rows, cudaStream_t stream) {
    const int vecs = p.d * (KIND == kReadF32 ? 4 : 2) / 16;  // 1 .. 64
    if (vecs <= 8) return launch_read_lanes<KIND, 8>(p, rows, stream);
    if (vecs <= 16) return launch_read_lanes<KIND, 16>(p, rows, stream);
    if (vecs <= 32) return launch_read_lanes<KIND, 32>(p, rows, stream);
    return launch_read_lanes<KIND, 64>(p, rows, stream);
}

}  // namespace

cudaError_t launch_append_q4(const AppendParams& p, int max_n_new, cudaStream_t stream) {
    const int vecs = p.row_bytes / 16;  // 4 .. 32
    if (vecs <= 4) return launch_append_lanes<4>(p, max_n_new, stream);
    if (vecs <= 8) return launch_append_lanes<8>(p, max_n_new, stream);
    if (vecs <= 16) return launch_append_lanes<16>(p, max_n_new, stream);
    return launch_append_lanes<32>(p, max_n_new, stream);
}

cudaError_t launch_read_rows(const ReadParams& p, int max_count, cudaStream_t stream) {
    switch (p.kind) {
        case kReadF32: return launch_read_kind<kReadF32>(p, max_count, stream);
        case kReadBf16: return launch_read_kind<kReadBf16>(p, max_count, stream);
        case kReadFp8: return launch_read_kind<kReadFp8>(p, max_count, stream);
        case kReadQ4: return launch_read_kind<kReadQ4>(p, max_count, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace kvc
