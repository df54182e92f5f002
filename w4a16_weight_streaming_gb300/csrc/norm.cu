// What stands between two blocks of a decoder, in one pass over the rows:
//
//   z = y                                                     the block's output, or its own norm
//       y * (1 / sqrt(mean(y^2) + eps)) * (offset + post)     (a norm behind the block)
//   h' = h + scale * gate * z                                 the residual stream, fp16 or fp32
//   x  = h' * (1 / sqrt(mean(h'^2) + eps)) * (offset + w)     the norm before the next block
//
// All of it in binary32 from the stored values; h' and x are rounded once each, and x is the norm of the
// sum before its rounding (1 / sqrt is rsqrtf, within 2^-22 of itself). A row stays in the registers of the threads
// that loaded it: one read of y, h and the gate, one write of h' and x, two sums over the row between them. Sums: 8
// neighbours of a vector in pairs, a thread's vectors in turn, then the warp and the warps in a fixed order.
//
// Measured on one GB300 (rows of 5120, in a CUDA graph): 8192 rows with a norm behind the block and a gate for every
// element 65.0 us (419 MB, 6.45 TB/s, 0.95 of the measured copy), 1024 rows with an fp32 residual stream 9.7 us
// (6.5 TB/s, 0.96): memory. 64 rows 2.8 us, one row 2.6: the latency of a launch, a round of loads and two sums (0.2 of it
// the norms' weights, which are loaded with the rest: a call before the last may still be writing them when this one
// starts). Scalar fp32 with divisions and square roots for the two factors took 71.8 us for 8192 rows, 10.2 for 1024.
//
// Error of a factor: a sum of squares goes through 20 roundings of 2^-24 at most (4 in a vector's pairs and 1 to join them, 3 more
// vectors, 5 in the warp, 5 among warps, 2 for mean and eps), half of that after the root, rsqrtf 2^-22, 4 in the products: below 2^-19.
#include "common.cuh"
#include "internal.h"

namespace w4a16 {
namespace {

struct NormArgs {
    const unsigned char* h;  // fp16 or fp32 rows, NULL never
    const uint16_t* y;       // NULL: no block output, x is the norm of h
    const uint16_t* post;    // NULL: no norm behind the block
    const uint16_t* gate;    // NULL: none
    const uint16_t* weight;  // NULL: ones
    unsigned char* h_out;    // NULL: not written
    uint16_t* x;             // NULL: not written
    int64_t h_stride, y_stride, gate_stride;
    int M, H, gate_per_row;
    float scale, offset, eps, inv_h;
};

__device__ __forceinline__ uint4 ldg_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// A vector as four pairs of fp32.
using Pairs = unsigned long long[4];
__device__ __forceinline__ void to_f32(const uint4& v, Pairs& f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[i] = pack_f2(p.x, p.y);
    }
}
__device__ __forceinline__ uint4 to_f16(const Pairs& f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack_f2(f[i], lo, hi);
        const __half2 p = __floats2half2_rn(lo, hi);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float sum_squares(const Pairs& f) {
    unsigned long long s = mul_f2(f[0], f[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s = fma_f2(f[i], f[i], s);
    float lo, hi;
    unpack_f2(s, lo, hi);
    return lo + hi;
}

// Sum over the threads of a row: a warp, or all warps of the CTA through `part`.
template <bool WARP_ROW>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (WARP_ROW) return v;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Registers a thread. Where a CTA has one of many rows, more CTAs an SM are worth a few spilled registers (8192 rows of 5120,
// fp16: 40 65.0 us, 48 64.1, 56 67.7; 4096 rows of 7168: 43.0, 48.5, 47.1; four vectors, 2048 rows of 16384: 64 52.7, 128
// 59.4; with an fp32 stream two vectors, 8192 rows of 5120: 48 109, 64 78.3; four, 2048 rows of 16384: 64 105, 128 82.9).
// Wider rows take 1024 threads and spill: 2048 rows of 32768 136.5 us (fp16, 3.9 TB/s) and 226 (fp32, 3.6 TB/s).
template <int V, int THREADS, bool F32>
constexpr int registers_for() {
    return THREADS == 1024 ? 64 : THREADS == 512 ? (V == 2 ? (F32 ? 64 : 40) : (F32 ? 128 : 64)) : 128;
}

// V vectors of 8 elements a thread. WARP_ROW: a warp a row (4 a CTA of THREADS = 128), else a CTA of up to
// THREADS a row.
template <int V, bool WARP_ROW, int THREADS, bool F32>
__global__ void __maxnreg__((registers_for<V, THREADS, F32>())) block_norm_kernel(const NormArgs a, unsigned* status) {
    __shared__ float part[2][32];
    const int nt = WARP_ROW ? 32 : static_cast<int>(blockDim.x);
    const int t = WARP_ROW ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
    const int64_t m = WARP_ROW ? blockIdx.x * 4LL + (threadIdx.x >> 5) : blockIdx.x;
    griddep_launch_dependents();
    if (m >= a.M) return;
    constexpr bool kLate = THREADS == 512 && !F32;  // the next norm's weights when the sums' registers are free
    const int vecs = a.H / 8;
    griddep_wait();  // before any load: a norm's weights may be an earlier kernel's output as well
    uint4 pw[V], nw[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = t + i * nt;
        pw[i] = nw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (v < vecs && a.post) pw[i] = *reinterpret_cast<const uint4*>(a.post + 8 * v);
        if (!kLate && v < vecs && a.weight) nw[i] = *reinterpret_cast<const uint4*>(a.weight + 8 * v);
    }
    uint4 hv[V][F32 ? 2 : 1], yv[V], gv[V];
    const unsigned char* hrow = a.h + m * a.h_stride * (F32 ? 4 : 2);
    float per_row = a.scale;
    if (a.gate && a.gate_per_row) per_row *= __half2float(__ushort_as_half(a.gate[m * a.gate_stride]));
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = t + i * nt;
        hv[i][0] = yv[i] = gv[i] = make_uint4(0u, 0u, 0u, 0u);
        if (F32) hv[i][F32 ? 1 : 0] = make_uint4(0u, 0u, 0u, 0u);
        if (v >= vecs || !in_bounds(8 * v + 8 <= a.H && m < a.M, status)) continue;
        hv[i][0] = ldg_once(hrow + static_cast<int64_t>(v) * (F32 ? 32 : 16));
        if (F32) hv[i][F32 ? 1 : 0] = ldg_once(hrow + static_cast<int64_t>(v) * 32 + 16);
        if (a.y) yv[i] = ldg_once(a.y + m * a.y_stride + 8 * v);
        if (a.gate && !a.gate_per_row) gv[i] = *reinterpret_cast<const uint4*>(a.gate + m * a.gate_stride + 8 * v);
    }
    float r = 1.f;
    if (a.post) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            Pairs f;
            to_f32(yv[i], f);
            s += sum_squares(f);
        }
        r = rsqrtf(fmaf(row_sum<WARP_ROW>(s, part[0]), a.inv_h, a.eps));
    }
    const unsigned long long r2 = pack_f2(r, r), scale2 = pack_f2(per_row, per_row), offset2 = pack_f2(a.offset, a.offset);
    Pairs sum[V];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (F32) {
            const uint4 lo = hv[i][0], hi = hv[i][F32 ? 1 : 0];
            const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[i][j] = pack_f2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
        } else {
            to_f32(hv[i][0], sum[i]);
        }
        if (a.y) {
            Pairs f, g;
            to_f32(yv[i], f);
            if (a.post) {
                to_f32(pw[i], g);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = mul_f2(mul_f2(f[j], r2), add_f2(offset2, g[j]));
            }
            if (a.gate && !a.gate_per_row) {
                to_f32(gv[i], g);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = mul_f2(f[j], g[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[i][j] = fma_f2(scale2, f[j], sum[i][j]);
        }
        const int v = t + i * nt;
        if (a.h_out && v < vecs && in_bounds(8 * v + 8 <= a.H, status)) {
            unsigned char* o = a.h_out + (m * a.H + 8 * static_cast<int64_t>(v)) * (F32 ? 4 : 2);
            if (F32) {
                reinterpret_cast<ulonglong2*>(o)[0] = make_ulonglong2(sum[i][0], sum[i][1]);
                reinterpret_cast<ulonglong2*>(o)[1] = make_ulonglong2(sum[i][2], sum[i][3]);
            } else {
                *reinterpret_cast<uint4*>(o) = to_f16(sum[i]);
            }
        }
        if (v < vecs) s += sum_squares(sum[i]);
    }
    if (!a.x) return;
    if (kLate && a.weight) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (t + i * nt < vecs) nw[i] = *reinterpret_cast<const uint4*>(a.weight + 8 * (t + i * nt));
    }
    const float q = rsqrtf(fmaf(row_sum<WARP_ROW>(s, part[1]), a.inv_h, a.eps));
    const unsigned long long q2 = pack_f2(q, q);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = t + i * nt;
        if (v >= vecs || !in_bounds(8 * v + 8 <= a.H, status)) continue;
        Pairs f, g;
        to_f32(nw[i], g);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = mul_f2(sum[i][j], q2);
        if (a.weight) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = mul_f2(f[j], add_f2(offset2, g[j]));
        }
        *reinterpret_cast<uint4*>(a.x + m * a.H + 8 * static_cast<int64_t>(v)) = to_f16(f);
    }
}

template <int V, bool WARP_ROW, int THREADS>
cudaError_t launch_v(const NormArgs& a, bool f32, int threads, cudaStream_t s, unsigned* status) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(WARP_ROW ? (a.M + 3) / 4 : a.M), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return f32 ? cudaLaunchKernelEx(&cfg, block_norm_kernel<V, WARP_ROW, THREADS, true>, a, status)
               : cudaLaunchKernelEx(&cfg, block_norm_kernel<V, WARP_ROW, THREADS, false>, a, status);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormParams& p, int sm_count, cudaStream_t s, unsigned* status) {
    const NormArgs a = {static_cast<const unsigned char*>(p.h), p.y, p.post, p.gate, p.weight, static_cast<unsigned char*>(p.h_out), p.x,
                        p.h_stride, p.y_stride, p.gate_stride, p.M, p.H, p.gate_per_row, p.scale, p.offset, p.eps, 1.f / static_cast<float>(p.H)};
    const bool f32 = p.h_f32 != 0;
    const int vecs = p.H / 8;
    if (vecs <= 32) return launch_v<1, true, 128>(a, f32, 128, s, status);
    if (vecs <= 64) return launch_v<2, true, 128>(a, f32, 128, s, status);
    if (vecs <= 128 && p.M > sm_count) return launch_v<4, true, 128>(a, f32, 128, s, status);
    auto threads = [&](int v) { return ((vecs + v - 1) / v + 31) / 32 * 32; };
    // Few rows: a vector a thread, the shortest way through a row. Many: two (8192 rows of 5120, with the registers not
    // limited: one 89 us, two 71.6, four 77.8, eight 129), four where that is too many threads.
    const bool few = p.M <= 2 * sm_count;
    if (!few && threads(2) <= 512) return launch_v<2, false, 512>(a, f32, threads(2), s, status);
    if (!few && threads(4) <= 512) return launch_v<4, false, 512>(a, f32, threads(4), s, status);
    if (threads(1) <= 1024) return launch_v<1, false, 1024>(a, f32, threads(1), s, status);
    if (threads(2) <= 1024) return launch_v<2, false, 1024>(a, f32, threads(2), s, status);
    return launch_v<4, false, 1024>(a, f32, threads(4), s, status);  // H <= 32768
}

}  // namespace w4a16
