// Attention over the 4-bit paged key/value cache: o = softmax(scale q k'^T) v' with k', v' the stored
// values min + code * scale. One CTA per (query row, query head); each warp takes tokens in turn with a
// running maximum and sum, the four warps are joined at the end.
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace w4a16 {
namespace {

template <int D>
__global__ void __launch_bounds__(128) kv4_attention_kernel(const Kv4AttnParams p, const Kv4View cache,
                                                            unsigned* status) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int L = D / 8, P = 32 / L;  // lanes per token, tokens per warp and step
    using T = Kv4<D>;
    const int row = blockIdx.x, head = blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __shared__ int s_seq;
    if (threadIdx.x == 0) s_seq = -1;
    __syncthreads();
    for (int b = threadIdx.x; b < p.B; b += 128)
        if (p.q_start[b] <= row && row < p.q_start[b + 1]) s_seq = b;
    __syncthreads();
    const int b = s_seq;
    if (b < 0) return;
    const int kvh = head / (p.heads / cache.kv_heads);
    const int len = p.kv_len[b], n = min(max(len, 0), p.max_pages << cache.page_shift);
    const int q_end = min(p.q_start[b + 1], p.M);
    if (len != n || q_end != p.q_start[b + 1]) record_error(status, kErrBounds);
    const int vis = p.causal ? min(n, n - (q_end - row) + 1) : n;
    const int d0 = (lane % L) * 8;
    float q[8], acc[8] = {};
    {
        const __half* src = reinterpret_cast<const __half*>(p.q) + row * p.q_stride + static_cast<int64_t>(head) * D + d0;
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __half2float(src[i]) * p.scale;
    }
    float mx = -INFINITY, sum = 0.f;
    for (int t0 = warp * P; t0 < vis; t0 += 4 * P) {
        const int tok = t0 + lane / L;
        float sc = 0.f;
        const uint8_t* tile = nullptr;
        const int page = tok < vis ? p.block_table[static_cast<int64_t>(b) * p.max_pages + (tok >> cache.page_shift)] : -1;
        const bool ok = page >= 0 && page < cache.num_pages;
        if (tok < vis && !ok) record_error(status, kErrBounds);
        const int in_page = tok & ((1 << cache.page_shift) - 1), tk = tok & 15, y = d0 / kKv4Group;
        if (ok) {
            tile = cache.pages + cache.tile_offset<D>(page, kvh, in_page);
            const float2 kp = __half22float2(*reinterpret_cast<const __half2*>(tile + T::k_param(tk, y)));
            const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + T::k_word(tk, d0));
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sc = fmaf(q[i], fmaf(static_cast<float>((w >> (4 * (i / 2 + 4 * (i & 1)))) & 15u), kp.x, kp.y), sc);
        }
#pragma unroll
        for (int o = 1; o < L; o <<= 1) sc += __shfl_xor_sync(0xffffffffu, sc, o);
        if (!ok) continue;
        const float nm = fmaxf(mx, sc);
        const float f = mx == -INFINITY ? 0.f : expf(mx - nm), e = expf(sc - nm);
        const float2 vp = __half22float2(*reinterpret_cast<const __half2*>(tile + T::v_param(tk, y)));
        mx = nm;
        sum = sum * f + e;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = fmaf(static_cast<float>((tile[T::v_byte(tk, d0 / 16, i)] >> ((d0 & 8) ? 4 : 0)) & 15u), vp.x, vp.y);
            acc[i] = fmaf(e, v, acc[i] * f);
        }
    }
    __shared__ float s_acc[4 * P][D], s_m[4 * P], s_l[4 * P];
    const int part = warp * P + lane / L;
#pragma unroll
    for (int i = 0; i < 8; ++i) s_acc[part][d0 + i] = acc[i];
    if (d0 == 0) {
        s_m[part] = mx;
        s_l[part] = sum;
    }
    __syncthreads();
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < 4 * P; ++i) m = fmaxf(m, s_m[i]);
    for (int i = 0; i < 4 * P; ++i) l += s_m[i] == -INFINITY ? 0.f : s_l[i] * expf(s_m[i] - m);
    for (int d = threadIdx.x; d < D; d += 128) {
        float o = 0.f;
        for (int i = 0; i < 4 * P; ++i) o += s_m[i] == -INFINITY ? 0.f : s_acc[i][d] * expf(s_m[i] - m);
        reinterpret_cast<__half*>(p.out)[(static_cast<int64_t>(row) * p.heads + head) * D + d] =
            __float2half_rn(l > 0.f ? o / l : 0.f);
    }
    if (p.lse != nullptr && threadIdx.x == 0)
        p.lse[static_cast<int64_t>(row) * p.heads + head] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t kv4_attention_workspace(int) { return 256; }

cudaError_t launch_kv4_attention(const Kv4AttnParams& p, const Kv4Cache& c, int sm_count, cudaStream_t s,
                                 unsigned* status) {
    (void)sm_count;
    Kv4View v;
    v.pages = static_cast<uint8_t*>(c.pages);
    v.num_pages = c.num_pages;
    v.page_shift = 0;
    while ((1 << v.page_shift) < c.page_tokens) ++v.page_shift;
    v.kv_heads = c.kv_heads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.M), static_cast<unsigned>(p.heads), 1);
    cfg.blockDim = dim3(128, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    switch (c.head_dim) {
        case 64: return cudaLaunchKernelEx(&cfg, kv4_attention_kernel<64>, p, v, status);
        case 128: return cudaLaunchKernelEx(&cfg, kv4_attention_kernel<128>, p, v, status);
        default: return cudaLaunchKernelEx(&cfg, kv4_attention_kernel<256>, p, v, status);
    }
}

}  // namespace w4a16
