// Writing and reading the 4-bit paged key/value cache.
//
// Append: one fused row holds the query, key and value heads of a token (the output of the qkv product).
// A head's D elements belong to D / 8 lanes, 8 consecutive elements (16 bytes) a lane, so that
//   - the sum of squares of a head's norm is 8 additions in a lane and log2(D / 8) exchanges,
//   - the rotation's partner element is in the same lane (adjacent pairs) or one exchange away (halves),
//   - the minimum and maximum of the 64 elements that share a scale are 3 exchanges among 8 lanes,
// and one pass takes a row from the product's output to rotated queries and stored codes. A decode row is
// bound by latency (a load, three short exchange chains, a store). A prompt chunk is near no single limit: 318
// instructions a warp for 256 elements at 2.6 of 4 a cycle, 46 % of the warps there, the first stall the first
// wave's loads. Rows are the grid's first dimension, so no thread divides (1024 rows 15.2 us with one index over
// rows and heads, 13.0 so).
//
// Measured with the reading kernel behind it, on one GB300, the data in L2: 1 row of 20 + 2 x 4 heads of 256
// 3.6 us the pair, 64 rows of 40 + 2 x 8 heads of 128 4.2 us, 1024 rows of 20 + 2 x 4 heads of 256 12.9 us (32
// MB in and out: 2.5 TB/s, 0.36 of the copy bandwidth).
//
// The codes are decisions, so everything before them is defined to the bit, in binary32 without fused
// multiply-adds: squares added 8 neighbours in turn, then sums of neighbours in pairs;
// y = (x * (1 / sqrt(sum / D + eps))) * w; (a, b) -> (a c - b s, b c + a s); one rounding to fp16; then
//   scale = fp16((max - min) / 15), code = rne((x - min) / scale) clamped to 0..15, 0 where scale is 0.
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace w4a16 {
namespace {

struct AppendArgs {
    const uint16_t* qkv;
    int64_t qkv_stride;  // elements between rows
    uint16_t* q_out;     // [M][heads][D], or null when heads is 0
    Kv4View cache;
    const int32_t* slots;
    const int32_t* positions;
    const float* rope;  // [rope_positions][rot]: rot / 2 cosines, rot / 2 sines; null: no rotation
    int rope_positions;
    int rot;
    int adjacent;
    const uint16_t* q_norm;  // [D] fp16 or null
    const uint16_t* k_norm;
    float eps;
    int M;
    int heads;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(const AppendArgs a, unsigned* status) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int L = D / 8;  // lanes per head
    using T = Kv4<D>;
    const int lane = threadIdx.x & 31;
    const int l = lane % L;
    const int d0 = l * 8;
    const int per_row = a.heads + 2 * a.cache.kv_heads;
    const int64_t m = blockIdx.x;
    const int slot_head = static_cast<int>((blockIdx.y * blockDim.x + threadIdx.x) / L);
    const bool live = slot_head < per_row;  // every lane takes part in the exchanges
    const int head = live ? slot_head : 0;
    const bool is_q = head < a.heads;
    const bool is_k = !is_q && head < a.heads + a.cache.kv_heads;

    uint4 raw = make_uint4(0, 0, 0, 0);
    if (live && in_bounds(m * a.qkv_stride + static_cast<int64_t>(head) * D + d0 + 8 <=
                              static_cast<int64_t>(a.M - 1) * a.qkv_stride + static_cast<int64_t>(per_row) * D,
                          status))
        raw = *reinterpret_cast<const uint4*>(a.qkv + m * a.qkv_stride + static_cast<int64_t>(head) * D + d0);
    // what the row and its position bring, asked for with the row itself
    const uint16_t* norm = is_q ? a.q_norm : is_k ? a.k_norm : nullptr;
    uint4 norm_raw = make_uint4(0, 0, 0, 0);
    if (norm != nullptr) norm_raw = *reinterpret_cast<const uint4*>(norm + d0);
    const int position = a.rope != nullptr ? a.positions[m] : 0;
    const int64_t slot = is_q ? -1 : a.slots[m];
    float x[8];
    unpack8(raw, x);

    bool ok = live;
    // A warp's lanes may belong to heads of different kinds (D < 256): all take part in the exchanges.
    float s = __fmul_rn(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) s = __fadd_rn(s, __fmul_rn(x[i], x[i]));
#pragma unroll
    for (int o = 1; o < L; o <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
    if (norm != nullptr) {
        // (s / D and 1 / sqrt, rounded as the divisions are)
        const float inv = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(s, 1.f / D), a.eps)));
        float w[8];
        unpack8(norm_raw, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], inv), w[i]);
    }
    int pos = 0;
    if (a.rope != nullptr && live) {
        pos = position;
        if (pos < 0 || pos >= a.rope_positions) {  // no such row of the table: nothing is stored
            if (l == 0) record_error(status, kErrBounds);
            ok = false;
            pos = 0;
        }
    }
    if (a.rope != nullptr) {
        const int half = a.rot / 2;
        const float* row = a.rope + static_cast<int64_t>(pos) * a.rot;
        if (a.adjacent) {
            if ((is_q || is_k) && d0 < a.rot) {
                const float4 c = *reinterpret_cast<const float4*>(row + d0 / 2);
                const float4 s = *reinterpret_cast<const float4*>(row + half + d0 / 2);
                const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float u = x[2 * i], v = x[2 * i + 1];
                    x[2 * i] = __fsub_rn(__fmul_rn(u, cc[i]), __fmul_rn(v, ss[i]));
                    x[2 * i + 1] = __fadd_rn(__fmul_rn(v, cc[i]), __fmul_rn(u, ss[i]));
                }
            }
        } else {
            const bool first = d0 < half;
            const bool turn = (is_q || is_k) && d0 < a.rot;
            const int src = turn ? (first ? lane + half / 8 : lane - half / 8) : lane;
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], src);
            if (turn) {
                const float* cs = row + (first ? d0 : d0 - half);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float4 c = *reinterpret_cast<const float4*>(cs + 4 * q);
                    const float4 s = *reinterpret_cast<const float4*>(cs + half + 4 * q);
                    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int e = 4 * q + i;
                        x[e] = first ? __fsub_rn(__fmul_rn(x[e], cc[i]), __fmul_rn(y[e], ss[i]))
                                     : __fadd_rn(__fmul_rn(x[e], cc[i]), __fmul_rn(y[e], ss[i]));
                    }
                }
            }
        }
    }
    uint4 packed = pack8(x);
    if (is_q) {
        if (live) {
            if (!ok) packed = make_uint4(0, 0, 0, 0);
            if (in_bounds((m * a.heads + head) * D + d0 + 8 <= static_cast<int64_t>(a.M) * a.heads * D, status))
                *reinterpret_cast<uint4*>(a.q_out + (m * a.heads + head) * D + d0) = packed;
        }
    }
    if (__all_sync(0xffffffffu, is_q || !live)) return;
    // ---- keys and values: the fp16 values above, in 4 bits (query lanes of a mixed warp run along)
    unpack8(packed, x);
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const __half scale = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
    const float sf = __half2float(scale);
    // (x - min) / scale, correctly rounded: a quotient by the rounded reciprocal and one correction (Markstein
    // 1990), 3 instructions an element instead of a division each
    const float inv_sf = sf > 0.f ? __frcp_rn(sf) : 0.f;
    uint32_t code[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = __fsub_rn(x[i], lo), quotient = __fmul_rn(a, inv_sf);
        const float c = rintf(__fmaf_rn(__fmaf_rn(-quotient, sf, a), inv_sf, quotient));
        code[i] = static_cast<uint32_t>(fminf(fmaxf(c, 0.f), 15.f));
    }
    uint32_t seq = 0;  // code i in nibble i
#pragma unroll
    for (int i = 0; i < 8; ++i) seq |= code[i] << (4 * i);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, seq, 1);
    if (is_q || !ok) return;

    if (slot < 0) return;  // a padding row: nothing is stored
    if (slot >= a.cache.slots()) {
        if (l == 0) record_error(status, kErrBounds);
        return;
    }
    const int kvh = head - a.heads - (is_k ? 0 : a.cache.kv_heads);
    const int in_page = static_cast<int>(slot) & ((1 << a.cache.page_shift) - 1);
    const int64_t off = a.cache.tile_offset<D>(static_cast<int>(slot >> a.cache.page_shift), kvh, in_page);
    if (!in_bounds(off >= 0 && off + T::kTileBytes <= a.cache.bytes<D>(), status)) return;
    uint8_t* tile = a.cache.pages + off;
    const int tk = in_page & 15;
    const int y = d0 / kKv4Group;
    if (is_k) {
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) word |= code[i] << (4 * (i / 2 + 4 * (i & 1)));
        *reinterpret_cast<uint32_t*>(tile + T::k_word(tk, d0)) = word;
    } else {
        const uint32_t low = (l & 1) ? other : seq, high = (l & 1) ? seq : other;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int g = (l & 1) * 4 + i;
            tile[T::v_byte(tk, d0 / 16, g)] =
                static_cast<uint8_t>(((low >> (4 * g)) & 15u) | (((high >> (4 * g)) & 15u) << 4));
        }
    }
    if ((l & 7) == 0) {
        const __half2 p = __halves2half2(scale, __float2half_rn(lo));
        *reinterpret_cast<__half2*>(tile + (is_k ? T::k_param(tk, y) : T::v_param(tk, y))) = p;
    }
}

// Load: the stored values of the tokens in `slots`, as fp16 (one rounding of min + code * scale). The
// same lanes as above; a negative slot gives zeros. A trip to the slots and one to the tile, so latency: 1024
// tokens of 4 heads of 256 cold 6.2 us (4.2 MB written).
template <int D>
__global__ void __launch_bounds__(256) kv4_load_kernel(const Kv4View cache, const int32_t* __restrict__ slots,
                                                       uint16_t* __restrict__ k, uint16_t* __restrict__ v, int n,
                                                       unsigned* status) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int L = D / 8;
    using T = Kv4<D>;
    const int d0 = static_cast<int>(threadIdx.x % L) * 8;
    const int64_t row = blockIdx.x;
    const int r = static_cast<int>((blockIdx.y * blockDim.x + threadIdx.x) / L);
    if (r >= 2 * cache.kv_heads) return;
    const bool is_k = r < cache.kv_heads;
    const int head = is_k ? r : r - cache.kv_heads;
    const int64_t slot = slots[row];
    float x[8] = {};
    if (slot >= cache.slots()) {
        if (d0 == 0) record_error(status, kErrBounds);
    } else if (slot >= 0) {
        const int in_page = static_cast<int>(slot) & ((1 << cache.page_shift) - 1);
        const int64_t off = cache.tile_offset<D>(static_cast<int>(slot >> cache.page_shift), head, in_page);
        if (in_bounds(off >= 0 && off + T::kTileBytes <= cache.bytes<D>(), status)) {
            const uint8_t* tile = cache.pages + off;
            const int tk = in_page & 15, y = d0 / kKv4Group;
            const float2 p = __half22float2(
                *reinterpret_cast<const __half2*>(tile + (is_k ? T::k_param(tk, y) : T::v_param(tk, y))));
            if (is_k) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + T::k_word(tk, d0));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i] = fmaf(static_cast<float>((w >> (4 * (i / 2 + 4 * (i & 1)))) & 15u), p.x, p.y);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i] = fmaf(static_cast<float>((tile[T::v_byte(tk, d0 / 16, i)] >> ((d0 & 8) ? 4 : 0)) & 15u), p.x,
                                p.y);
            }
        }
    }
    uint16_t* out = is_k ? k : v;
    if (in_bounds((row * cache.kv_heads + head) * D + d0 + 8 <= static_cast<int64_t>(n) * cache.kv_heads * D, status))
        *reinterpret_cast<uint4*>(out + (row * cache.kv_heads + head) * D + d0) = pack8(x);
}

template <typename F, typename... A>
cudaError_t launch_rows(F* f, int rows, int heads, int lanes, cudaStream_t s, A... args) {
    // a grid row of CTAs a token, its heads dealt evenly to as few CTAs of up to 256 threads as hold them
    const int parts = (heads * lanes + 255) / 256, threads = ((heads + parts - 1) / parts * lanes + 31) / 32 * 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows), static_cast<unsigned>(parts), 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, f, args...);
}

Kv4View view(const Kv4Cache& c) {
    Kv4View v;
    v.pages = static_cast<uint8_t*>(c.pages);
    v.num_pages = c.num_pages;
    v.page_shift = 0;
    while ((1 << v.page_shift) < c.page_tokens) ++v.page_shift;
    v.kv_heads = c.kv_heads;
    return v;
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendParams& p, const Kv4Cache& c, cudaStream_t s, unsigned* status) {
    AppendArgs a;
    a.qkv = p.qkv;
    a.qkv_stride = p.qkv_stride;
    a.q_out = p.q_out;
    a.cache = view(c);
    a.slots = p.slots;
    a.positions = p.positions;
    a.rope = p.rope;
    a.rope_positions = p.rope_positions;
    a.rot = p.rot;
    a.adjacent = p.adjacent;
    a.q_norm = p.q_norm;
    a.k_norm = p.k_norm;
    a.eps = p.eps;
    a.M = p.M;
    a.heads = p.heads;
    const int heads = p.heads + 2 * c.kv_heads;
    switch (c.head_dim) {
        case 64: return launch_rows(kv4_append_kernel<64>, p.M, heads, 8, s, a, status);
        case 128: return launch_rows(kv4_append_kernel<128>, p.M, heads, 16, s, a, status);
        default: return launch_rows(kv4_append_kernel<256>, p.M, heads, 32, s, a, status);
    }
}

cudaError_t launch_kv4_load(const Kv4Cache& c, const int32_t* slots, uint16_t* k, uint16_t* v, int n, cudaStream_t s,
                            unsigned* status) {
    const Kv4View w = view(c);
    switch (c.head_dim) {
        case 64: return launch_rows(kv4_load_kernel<64>, n, 2 * c.kv_heads, 8, s, w, slots, k, v, n, status);
        case 128: return launch_rows(kv4_load_kernel<128>, n, 2 * c.kv_heads, 16, s, w, slots, k, v, n, status);
        default: return launch_rows(kv4_load_kernel<256>, n, 2 * c.kv_heads, 32, s, w, slots, k, v, n, status);
    }
}

}  // namespace w4a16
