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

// LANES: lanes a row (a power of two, d / 8 or more of them: the others idle).
template <int LANES>
__global__ void __launch_bounds__(kThreads) append_q4_kernel(const __grid_constant__ AppendParams p) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int b = blockIdx.z, h = blockIdx.y >> 1;
    const bool is_v = (blockIdx.y & 1) != 0;
    const int n = p.n_new[b];
    const int sub = threadIdx.x % LANES;
    const int t = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    if (blockIdx.x * (kThreads / LANES) >= n) return;
    const int vecs = p.row_bytes / 16;  // 16-byte vectors of a bf16 row
    const bool live = t < n && sub < vecs;
    const size_t unit = static_cast<size_t>(b) * p.Hkv + h;
    const uint8_t* src = (is_v ? p.v_new : p.k_new) + unit * p.T * p.row_bytes;
    uint4 val = make_uint4(0u, 0u, 0u, 0u);
    if (live) val = __ldg(reinterpret_cast<const uint4*>(src + static_cast<size_t>(t) * p.row_bytes) + sub);
    const uint32_t w[4] = {val.x, val.y, val.z, val.w};
    float lo, hi;
    q4::range8(w, lo, hi);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (!live) return;
    const q4::RowScale rs = q4::row_scale(lo, hi);
    bool bad = false;  // (a position whose block-table entry is bad is not written)
    const int row = phys_row(p.pg, p.ring, p.Hkv, p.max_len, b, h, p.lens[b] + t, &bad);
    if (bad) return;
    uint32_t* codes = reinterpret_cast<uint32_t*>(is_v ? p.v_cache : p.k_cache);
    codes[static_cast<size_t>(row) * vecs + sub] = q4::encode8(w, rs);
    if (sub == 0) (is_v ? p.q4.v : p.q4.k)[q4::scale_index(p.q4, row)] = rs.word;
}

// KIND as in ReadParams.
template <int KIND>
__global__ void __launch_bounds__(kThreads) read_rows_kernel(const __grid_constant__ ReadParams p) {
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int b = blockIdx.z, h = blockIdx.y >> 1;
    const bool is_v = (blockIdx.y & 1) != 0;
    const int vecs = p.d * (KIND == kReadF32 ? 4 : 2) / 16;  // 16-byte vectors of a result row
    const long long vec = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    if (vec >= static_cast<long long>(p.count[b]) * vecs) return;
    const int t = static_cast<int>(vec / vecs), c = static_cast<int>(vec - static_cast<long long>(t) * vecs);
    bool bad = false;  // a bad block-table entry reads as zeros
    const int row = phys_row(p.pg, p.ring, p.Hkv, p.max_len, b, h, p.first[b] + t, &bad);
    const uint8_t* cache = is_v ? p.v_cache : p.k_cache;
    uint32_t o[4] = {0u, 0u, 0u, 0u};
    if (!bad) {
        if constexpr (KIND == kReadQ4) {
            const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(cache) + static_cast<size_t>(row) * vecs + c);
            const uint32_t sw = __ldg((is_v ? p.q4.v : p.q4.k) + q4::scale_index(p.q4, row));
            const float s = q4::step_of(sw);
            const int z = q4::zero_of(sw);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = ptx::pack_bf16x2(s * static_cast<float>(q4::code_of(w, 2 * i) - z),
                                        s * static_cast<float>(q4::code_of(w, 2 * i + 1) - z));
        } else if constexpr (KIND == kReadFp8) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(cache) + static_cast<size_t>(row) * vecs + c);
            const float s = is_v ? p.vscale[h] : p.kscale[h];
            const uint32_t in[2] = {w.x, w.y};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t f[2];
                ptx::e4m3x4_to_f16x2x2(in[i], f[0], f[1]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    __half2 hh;
                    memcpy(&hh, &f[j], 4);
                    const float2 v = __half22float2(hh);
                    o[2 * i + j] = ptx::pack_bf16x2(v.x * s, v.y * s);
                }
            }
        } else {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(cache) + static_cast<size_t>(row) * vecs + c);
            o[0] = w.x, o[1] = w.y, o[2] = w.z, o[3] = w.w;
        }
    }
    const size_t unit = static_cast<size_t>(b) * p.Hkv + h;
    uint4* dst = reinterpret_cast<uint4*>(is_v ? p.v_out : p.k_out) + unit * p.T * vecs;
    dst[vec] = make_uint4(o[0], o[1], o[2], o[3]);
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

template <int LANES>
cudaError_t launch_append_lanes(const AppendParams& p, int max_n_new, cudaStream_t stream) {
    constexpr int rows = kThreads / LANES;
    const dim3 grid(static_cast<unsigned>((max_n_new + rows - 1) / rows), 2u * p.Hkv, p.B);
    return launch_chained(append_q4_kernel<LANES>, grid, stream, p);
}

}  // namespace

cudaError_t launch_append_q4(const AppendParams& p, int max_n_new, cudaStream_t stream) {
    const int vecs = p.row_bytes / 16;
    if (vecs <= 4) return launch_append_lanes<4>(p, max_n_new, stream);
    if (vecs <= 8) return launch_append_lanes<8>(p, max_n_new, stream);
    if (vecs <= 16) return launch_append_lanes<16>(p, max_n_new, stream);
    return launch_append_lanes<32>(p, max_n_new, stream);
}

cudaError_t launch_read_rows(const ReadParams& p, int max_count, cudaStream_t stream) {
    const long long vecs = static_cast<long long>(max_count) * (p.d * (p.kind == kReadF32 ? 4 : 2) / 16);
    const dim3 grid(static_cast<unsigned>((vecs + kThreads - 1) / kThreads), 2u * p.Hkv, p.B);
    switch (p.kind) {
        case kReadF32: return launch_chained(read_rows_kernel<kReadF32>, grid, stream, p);
        case kReadBf16: return launch_chained(read_rows_kernel<kReadBf16>, grid, stream, p);
        case kReadFp8: return launch_chained(read_rows_kernel<kReadFp8>, grid, stream, p);
        case kReadQ4: return launch_chained(read_rows_kernel<kReadQ4>, grid, stream, p);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace kvc
