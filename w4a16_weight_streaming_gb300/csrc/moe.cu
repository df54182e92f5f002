// A mixture-of-experts layer for a few tokens (T <= 64), its experts' weights in 4 bits:
//
//   l[t][e] = x[t] . router[e]                                     fp16 products, fp32 sums
//   score   = softmax_e(l) or sigmoid(l); chosen: the k experts with the largest l, or score + bias
//             (ties: the lower index); r[t][e] = score, over the sum of the chosen ones' if asked, times `scale`
//   a[t][e] = fp16(silu(x[t] . Wg[e]) * (x[t] . Wu[e]))            for the chosen e, products kept in fp32
//   y[t]    = fp16(sum_e r[t][e] * (a[t][e] . Wd[e]))              summed in order of e, in fp32
//
// Three kernels on one stream, each scheduled while the one before it runs:
//   route    a CTA per expert and 8 tokens; the last CTA of 8 tokens chooses their experts, the last of all
//            lists the experts that were chosen, each with its tokens
//   gate_up  a CTA per listed expert and 16 gate + 16 up columns over the whole of K
//   down     a CTA (or cluster) per 32 output columns over all listed experts: so the sum over the experts of
//            a token is made in one place and in one order, without atomics
//
// What bounds it is the weights of the chosen experts, read once each whatever the tokens. They go from
// global memory through registers into mma.m16n8k16 as the A operand (16 columns of W), tokens are its 8
// columns: a lane (g, t) = (lane / 4, lane % 4) takes the whole 16-byte vector of column g and 32-k block t of
// four adjacent blocks, so that of every 128 k a lane's loads are wide and dense and nothing is exchanged:
// the instruction's k slots are simply numbered so that lane t's are the k of its own block. The B operand
// must follow, so rows of x and of a are kept with their 16-byte units transposed within each 128 (unit w of
// block t at place 4 w + t).
#include "common.cuh"
#include "internal.h"

namespace w4a16 {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

// ------------------------------------------------------------------------------------ workspace
// The same layout for every call with the same experts.
struct Plan {  // what the router leaves to the other kernels
    int active;                       // listed experts
    int expert[kMoeMaxExperts];
    int base[kMoeMaxExperts + 1];     // of a listed expert's first (token, weight) pair
    int token[kMoeMaxTokens * kMoeMaxTop];
    float weight[kMoeMaxTokens * kMoeMaxTop];
};
struct Space {
    unsigned* arrived;  // 8 groups of 8 tokens, then the groups
    Plan* plan;
    int* chosen;        // [tokens][k]
    float* share;       // [tokens][k]
    float* logits;      // [tokens][E]
    uint16_t* xp;       // [tokens][Hp], transposed units
    uint16_t* act;      // [pairs][Ip], transposed units
    size_t bytes;
};

__host__ __device__ inline int64_t padded(int k) { return (static_cast<int64_t>(k) + 127) / 128 * 128; }

inline Space space_of(void* base, int E, int H, int I) {
    Space s;
    unsigned char* p = static_cast<unsigned char*>(base);
    size_t at = 0;
    auto take = [&](size_t n) {
        unsigned char* q = p + at;
        at += (n + 255) / 256 * 256;
        return q;
    };
    s.arrived = reinterpret_cast<unsigned*>(take(64));
    s.plan = reinterpret_cast<Plan*>(take(sizeof(Plan)));
    s.chosen = reinterpret_cast<int*>(take(kMoeMaxTokens * kMoeMaxTop * 4));
    s.share = reinterpret_cast<float*>(take(kMoeMaxTokens * kMoeMaxTop * 4));
    s.logits = reinterpret_cast<float*>(take(static_cast<size_t>(kMoeMaxTokens) * E * 4));
    s.xp = reinterpret_cast<uint16_t*>(take(kMoeMaxTokens * padded(H) * 2));
    s.act = reinterpret_cast<uint16_t*>(take(static_cast<size_t>(kMoeMaxTokens) * kMoeMaxTop * padded(I) * 2));
    s.bytes = at;
    return s;
}

// Place of element i of a row with transposed units.
__device__ __forceinline__ int64_t unit_place(int i) {
    return (static_cast<int64_t>(i) & ~127LL) + ((((i >> 3) & 3) * 4 + ((i >> 5) & 3)) << 3) + (i & 7);
}

__device__ __forceinline__ uint4 ldg_weights(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// ------------------------------------------------------------------------------------ routing
struct RouteArgs {
    const uint16_t* x;
    int64_t x_stride;
    const uint16_t* router;  // [E][H]
    const float* bias;       // [E] or NULL
    int32_t* ids;            // [T][k] or NULL
    float* weights;          // [T][k] or NULL
    Space w;
    int T, E, H, k, sigmoid, renormalize;
    float scale;
};

// A float as a whole number of the same order, above 1; NaN: 1 (below all).
__device__ __forceinline__ uint32_t order_of(float f) {
    if (f != f) return 1u;
    const uint32_t b = __float_as_uint(f + 0.f);  // -0 and 0 are one value
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// One warp chooses the experts of token t and their weights.
__device__ __forceinline__ void choose(const RouteArgs& a, int t) {
    constexpr int kEach = kMoeMaxExperts / 32;
    const int lane = threadIdx.x & 31;
    uint32_t key[kEach];
    float most = -INFINITY, all = 0.f;
    const float* row = a.w.logits + static_cast<int64_t>(t) * a.E;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        key[i] = 0;
        const int e = i * 32 + lane;
        if (i * 32 >= a.E || e >= a.E) continue;
        const float l = __ldcg(row + e);
        most = fmaxf(most, l);
        key[i] = order_of(a.sigmoid ? 1.f / (1.f + expf(-l)) + (a.bias ? a.bias[e] : 0.f) : l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (!a.sigmoid && !a.renormalize) {
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (i * 32 < a.E && i * 32 + lane < a.E) all += expf(__ldcg(row + i * 32 + lane) - most);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    int mine = 0;
    for (int r = 0; r < a.k; ++r) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (i * 32 < a.E) best = max(best, key[i]);
        best = __reduce_max_sync(0xffffffffu, best);
        uint32_t at = 0xFFFFFFFFu;
#pragma unroll
        for (int i = kEach - 1; i >= 0; --i)
            if (i * 32 < a.E && key[i] == best) at = static_cast<uint32_t>(i * 32 + lane);
        at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (static_cast<uint32_t>(i * 32 + lane) == at) key[i] = 0;
        if (lane == r) mine = static_cast<int>(at);
    }
    const float l = lane < a.k ? __ldcg(row + mine) : 0.f;
    float s = lane < a.k ? (a.sigmoid ? 1.f / (1.f + expf(-l)) : expf(l - most)) : 0.f;
    if (a.renormalize) {
        all = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    if (a.renormalize || !a.sigmoid) s = __fdiv_rn(s, fmaxf(all, 1e-30f));  // (sigmoids may all be 0)
    if (lane < a.k) {
        const int64_t at = static_cast<int64_t>(t) * a.k + lane;
        a.w.chosen[at] = mine;
        a.w.share[at] = s * a.scale;
        if (a.ids) a.ids[at] = mine;
        if (a.weights) a.weights[at] = s * a.scale;
    }
}

// The list of chosen experts with their tokens, by one CTA.
__device__ __forceinline__ void list_experts(const RouteArgs& a) {
    __shared__ uint32_t mask[2][kMoeMaxExperts];  // tokens of an expert, one bit each
    __shared__ uint32_t scan[kMoeMaxExperts];     // (listed experts << 16) + pairs, up to and with this one
    const int pairs = a.T * a.k;
    for (int e = threadIdx.x; e < kMoeMaxExperts; e += kThreads) mask[0][e] = mask[1][e] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += kThreads) {
        const int t = p / a.k;
        atomicOr(&mask[t >> 5][__ldcg(a.w.chosen + p)], 1u << (t & 31));
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kMoeMaxExperts; e += kThreads) {
        const uint32_t n = __popc(mask[0][e]) + __popc(mask[1][e]);
        scan[e] = n == 0 ? 0u : (1u << 16) + n;
    }
    __syncthreads();
    for (int o = 1; o < kMoeMaxExperts && o < a.E; o <<= 1) {
        uint32_t add[kMoeMaxExperts / kThreads];
#pragma unroll
        for (int i = 0; i < kMoeMaxExperts / kThreads; ++i) {
            const int e = static_cast<int>(threadIdx.x) + i * kThreads;
            add[i] = e >= o ? scan[e - o] : 0u;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kMoeMaxExperts / kThreads; ++i) scan[threadIdx.x + i * kThreads] += add[i];
        __syncthreads();
    }
    Plan* plan = a.w.plan;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        const uint32_t n = __popc(mask[0][e]) + __popc(mask[1][e]);
        if (n == 0) continue;
        const int at = static_cast<int>(scan[e] >> 16) - 1;
        plan->expert[at] = e;
        plan->base[at + 1] = static_cast<int>(scan[e] & 0xFFFFu);
    }
    if (threadIdx.x == 0) {
        plan->base[0] = 0;
        plan->active = static_cast<int>(scan[a.E - 1] >> 16);
    }
    for (int p = threadIdx.x; p < pairs; p += kThreads) {
        const int t = p / a.k, e = __ldcg(a.w.chosen + p);
        const uint32_t lo = mask[0][e], hi = mask[1][e], bit = 1u << (t & 31);
        const int before = t < 32 ? __popc(lo & (bit - 1)) : __popc(lo) + __popc(hi & (bit - 1));
        const int at = static_cast<int>(scan[e] & 0xFFFFu) - __popc(lo) - __popc(hi) + before;
        plan->token[at] = t;
        plan->weight[at] = __ldcg(a.w.share + p);
    }
}

// TB tokens a CTA (1 or 8), one expert.
template <int TB>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a, unsigned* status) {
    __shared__ float part[kWarps][TB];
    __shared__ int last;
    griddep_launch_dependents();
    const int e = blockIdx.x, group = blockIdx.y, t0 = group * TB;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tokens = min(TB, a.T - t0), vecs = a.H / 8;
    const uint16_t* wrow = a.router + static_cast<int64_t>(e) * a.H;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (static_cast<int>(threadIdx.x) < vecs) w = *reinterpret_cast<const uint4*>(wrow + 8 * threadIdx.x);
    griddep_wait();
    float acc[TB][2];
#pragma unroll
    for (int i = 0; i < TB; ++i) acc[i][0] = acc[i][1] = 0.f;
    for (int v = threadIdx.x; v < vecs; v += kThreads) {
        uint4 x[TB];
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            const int64_t at = (t0 + i) * a.x_stride + 8 * static_cast<int64_t>(v);
            x[i] = i < tokens && in_bounds(8 * v + 8 <= a.H, status) ? *reinterpret_cast<const uint4*>(a.x + at) : make_uint4(0u, 0u, 0u, 0u);
        }
        const int next = v + kThreads;
        const uint4 wn = next < vecs ? *reinterpret_cast<const uint4*>(wrow + 8 * next) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            fma2_mixed(acc[i][0], acc[i][1], w.x, x[i].x);
            fma2_mixed(acc[i][0], acc[i][1], w.y, x[i].y);
            fma2_mixed(acc[i][0], acc[i][1], w.z, x[i].z);
            fma2_mixed(acc[i][0], acc[i][1], w.w, x[i].w);
            if (e == 0 && i < tokens) {  // one expert's CTAs leave x as the products want it
                uint16_t* to = a.w.xp + (t0 + i) * padded(a.H) + unit_place(8 * v);
                *reinterpret_cast<uint4*>(to) = x[i];
            }
        }
        w = wn;
    }
#pragma unroll
    for (int i = 0; i < TB; ++i) {
        float s = acc[i][0] + acc[i][1];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) part[warp][i] = s;
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < tokens) {
        float s = part[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) s += part[i][threadIdx.x];
        a.w.logits[static_cast<int64_t>(t0 + threadIdx.x) * a.E + e] = s;
        __threadfence();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(a.w.arrived + group, 1u) == static_cast<unsigned>(a.E) - 1u;
        if (last) a.w.arrived[group] = 0;  // ready for the next call
        __threadfence();
    }
    __syncthreads();
    if (!last) return;
    for (int t = warp; t < tokens; t += kWarps) choose(a, t0 + t);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(a.w.arrived + 15, 1u) == gridDim.y - 1u;
        if (last) a.w.arrived[15] = 0;
        __threadfence();
    }
    __syncthreads();
    if (last) list_experts(a);
}

// ------------------------------------------------------------------------------------ products
struct Matrices {
    const uint4* w;       // repacked codes of all experts
    const uint16_t* s;    // repacked scales
    const float* factor;  // NVFP4: fp32 scale of each expert's matrix
    int N, K, G;          // of one expert
};

// D (16 columns x 8 tokens) += A (16 columns x 16 k) . B (16 k x 8 tokens)
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two bands of 16 columns of one expert's matrix, as a lane reads them: column g and g + 8 of each.
template <bool FP4>
struct Columns {
    const uint4* w[2];
    const uint16_t* s[2];
    int wt[2];     // vectors from one 32-k block to the next
    int blocks;    // 32-k blocks of K
    int shift, per;  // 32-k blocks a scale row (int4), as a shift where that is a power of two

    __device__ __forceinline__ void set(const Matrices& m, int expert, int c0, int c1, int lane) {
        blocks = m.K / 32;
        per = FP4 ? 1 : m.G / 32;
        shift = (per & (per - 1)) == 0 ? __ffs(per) - 1 : -1;
        const int rows = FP4 ? 2 * blocks : m.K / m.G;
        const int64_t codes = static_cast<int64_t>(expert) * m.N * blocks, scales = static_cast<int64_t>(expert) * m.N * rows;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int c = b ? c1 : c0, tile = c >> 7;
            wt[b] = min(128, m.N - 128 * tile);
            w[b] = m.w + codes + static_cast<int64_t>(tile) * 128 * blocks + (c & 127) + (lane >> 2);
            s[b] = m.s + scales + static_cast<int64_t>(tile) * 128 * rows + (c & 127) + (lane >> 2);
        }
    }
};

template <bool FP4>
struct Step {  // a lane's share of 128 k: 4 columns, 32 k each
    uint4 v[4];
    uint32_t s[4];  // int4: (scale, scale); NVFP4: (of the first 16 k, of the second)

    __device__ __forceinline__ void load(const Columns<FP4>& c, int kb, int lane, bool any) {
        const int blk = kb * 4 + (lane & 3);
        const bool there = any && blk < c.blocks;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint4* p = c.w[b] + static_cast<int64_t>(blk) * c.wt[b];
            v[2 * b] = there ? ldg_weights(p) : make_uint4(0u, 0u, 0u, 0u);
            v[2 * b + 1] = there ? ldg_weights(p + 8) : make_uint4(0u, 0u, 0u, 0u);
            if (FP4) {
                const uint16_t* q = c.s[b] + static_cast<int64_t>(2 * blk) * c.wt[b];
                s[2 * b] = there ? __ldg(q) | static_cast<uint32_t>(__ldg(q + c.wt[b])) << 16 : 0u;
                s[2 * b + 1] = there ? __ldg(q + 8) | static_cast<uint32_t>(__ldg(q + c.wt[b] + 8)) << 16 : 0u;
            } else {
                const int row = c.shift >= 0 ? blk >> c.shift : blk / c.per;
                const uint16_t* q = c.s[b] + static_cast<int64_t>(row) * c.wt[b];
                s[2 * b] = there ? __ldg(q) : 0u;
                s[2 * b + 1] = there ? __ldg(q + 8) : 0u;
            }
        }
    }

    // acc[b][n] += the bands' columns times NT * 8 tokens; rows[n]: this lane's token of those 8, NULL for none.
    template <int NT>
    __device__ __forceinline__ void multiply(float (&acc)[2][NT][4], const uint16_t* const (&rows)[NT], int tiles, int blocks, int kb,
                                             int lane) const {
        const bool there = kb * 4 + (lane & 3) < blocks;
        const int64_t at = (static_cast<int64_t>(kb) * 16 + (lane & 3)) * 8;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t d[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t word = w == 0 ? v[i].x : w == 1 ? v[i].y : w == 2 ? v[i].z : v[i].w;
                if (FP4) {
                    const uint32_t h = w < 2 ? s[i] & 0xFFFFu : s[i] >> 16;
                    dequant8_nvfp4(word, h * 0x10001u, d[i]);
                } else {
                    dequant8(word, s[i] * 0x10001u, d[i]);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n >= tiles) break;
                const uint4 x = there && rows[n] ? *reinterpret_cast<const uint4*>(rows[n] + at + w * 32) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    mma16816(acc[b][n], d[2 * b][0], d[2 * b + 1][0], d[2 * b][1], d[2 * b + 1][1], x.x, x.y);
                    mma16816(acc[b][n], d[2 * b][2], d[2 * b + 1][2], d[2 * b][3], d[2 * b + 1][3], x.z, x.w);
                }
            }
        }
    }
};

// CTA: listed expert blockIdx.x / chunks, gate columns 16 j .. and up columns I + 16 j .. The warps take the
// 128-k steps in turn and are added up through shared memory; SwiGLU on the sums.
template <int NT, bool FP4>
__global__ void __launch_bounds__(kThreads) gate_up_kernel(const Matrices m, const Space ws, int H, int I, unsigned* status) {
    __shared__ float2 red[kWarps][NT][2][64];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_wait();
    griddep_launch_dependents();  // (after the wait: the next kernel may read the plan before its own wait)
    const int chunks = I / 16;
    const int at = static_cast<int>(blockIdx.x) / chunks, j = static_cast<int>(blockIdx.x) % chunks;
    if (at >= __ldcg(&ws.plan->active)) return;
    const int expert = __ldcg(ws.plan->expert + at), base = __ldcg(ws.plan->base + at), count = __ldcg(ws.plan->base + at + 1) - base;
    const int steps = static_cast<int>(padded(H) / 128);
    Columns<FP4> cols;
    cols.set(m, expert, 16 * j, I + 16 * j, lane);
    for (int first = 0; first < count; first += 8 * NT) {
        const int tiles = min(NT, (count - first + 7) / 8);
        const uint16_t* rows[NT];
        float acc[2][NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int i = first + 8 * n + (lane >> 2);
            rows[n] = i < count ? ws.xp + __ldcg(ws.plan->token + base + i) * padded(H) : nullptr;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[b][n][r] = 0.f;
        }
        Step<FP4> cur, next;
        cur.load(cols, warp, lane, warp < steps);
        for (int kb = warp; kb < steps; kb += kWarps) {
            next.load(cols, kb + kWarps, lane, kb + kWarps < steps);
            cur.template multiply<NT>(acc, rows, tiles, cols.blocks, kb, lane);
            cur = next;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int b = 0; b < 2; ++b) {  // [column][token]
                red[warp][n][b][lane] = make_float2(acc[b][n][0], acc[b][n][1]);
                red[warp][n][b][32 + lane] = make_float2(acc[b][n][2], acc[b][n][3]);
            }
        __syncthreads();
        const float factor = FP4 ? m.factor[expert] : 1.f;
        for (int i = threadIdx.x; i < tiles * 128; i += kThreads) {
            // unit of 8 columns as consecutive threads, so that a row's stores are 16 bytes wide
            const int n = i >> 7, col = i & 15, tok = (i >> 4) & 7;
            const int pair = first + 8 * n + tok;
            if (pair >= count) continue;
            float sum[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const float* p = reinterpret_cast<const float*>(&red[0][n][b][0]) + col * 8 + tok;
                sum[b] = p[0];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) sum[b] += p[w * NT * 2 * 128];
                sum[b] *= factor;
            }
            const float act = sum[0] / (1.0f + expf(-sum[0])) * sum[1];
            if (in_bounds(base + pair < kMoeMaxTokens * kMoeMaxTop && 16 * j + col < I, status))
                ws.act[(base + pair) * padded(I) + unit_place(16 * j + col)] = __half_as_ushort(__float2half_rn(act));
        }
        __syncthreads();
    }
}

// CTA `rank` of a cluster of P: output columns 32 c .., the rank's share of all (listed expert, 128-k step) in
// order, each warp a run of it. Sums of a token are kept a warp in shared memory and added up in order.
template <int NT, bool FP4>
__global__ void __launch_bounds__(kThreads) down_kernel(const Matrices m, const Space ws, uint16_t* __restrict__ y, int T, int H, int I,
                                                        int P, unsigned* status) {
    extern __shared__ float total[];  // [warps][T][32], then [T][32] of the CTA
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_launch_dependents();
    const int rank = static_cast<int>(blockIdx.x) % P, chunk = static_cast<int>(blockIdx.x) / P;
    // The plan is the work of the kernel before the last: complete, since every CTA of the last one passed its wait
    // before this kernel could start.
    const int active = __ldcg(&ws.plan->active);
    const int steps = static_cast<int>(padded(I) / 128);
    const int runs = P * kWarps, run = rank * kWarps + warp, all = active * steps;
    int s = static_cast<int>(static_cast<int64_t>(all) * run / runs);
    const int end = static_cast<int>(static_cast<int64_t>(all) * (run + 1) / runs);
    float* mine = total + warp * T * 32;
    for (int i = lane; i < T * 32; i += 32) mine[i] = 0.f;
    int at = s / steps, kb = s % steps;
    Columns<FP4> cols;
    Step<FP4> cur, next;
    if (s < end) {
        cols.set(m, __ldcg(ws.plan->expert + at), 32 * chunk, 32 * chunk + 16, lane);
        cur.load(cols, kb, lane, true);
    }
    griddep_wait();
    __syncwarp();
    while (s < end) {
        const int base = __ldcg(ws.plan->base + at), count = __ldcg(ws.plan->base + at + 1) - base;
        const int stop = min(steps, kb + end - s);  // this expert's steps kb .. stop - 1
        const float factor = FP4 ? m.factor[__ldcg(ws.plan->expert + at)] : 1.f;
        const bool more = s + stop - kb < end;
        for (int first = 0; first < count; first += 8 * NT) {
            const int tiles = min(NT, (count - first + 7) / 8);
            const bool again = first + 8 * NT < count;
            const uint16_t* rows[NT];
            float acc[2][NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int i = first + 8 * n + (lane >> 2);
                rows[n] = i < count ? ws.act + (base + i) * padded(I) : nullptr;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[b][n][r] = 0.f;
            }
            for (int k = kb; k < stop; ++k) {
                if (k + 1 < stop) {
                    next.load(cols, k + 1, lane, true);
                } else if (again) {
                    next.load(cols, kb, lane, true);
                } else if (more) {
                    Columns<FP4> after;
                    after.set(m, __ldcg(ws.plan->expert + at + 1), 32 * chunk, 32 * chunk + 16, lane);
                    next.load(after, 0, lane, true);
                }
                cur.template multiply<NT>(acc, rows, tiles, cols.blocks, k, lane);
                cur = next;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int i = first + 8 * n + 2 * (lane & 3) + h;
                    if (i >= count) continue;
                    const int token = __ldcg(ws.plan->token + base + i);
                    const float w = __ldcg(ws.plan->weight + base + i) * factor;
                    if (!in_bounds(token >= 0 && token < T, status)) continue;
                    float* to = mine + token * 32 + (lane >> 2);
                    to[0] = fmaf(w, acc[0][n][h], to[0]);
                    to[8] = fmaf(w, acc[0][n][2 + h], to[8]);
                    to[16] = fmaf(w, acc[1][n][h], to[16]);
                    to[24] = fmaf(w, acc[1][n][2 + h], to[24]);
                }
            __syncwarp();
        }
        s += stop - kb;
        ++at;
        kb = 0;
        if (s < end) cols.set(m, __ldcg(ws.plan->expert + at), 32 * chunk, 32 * chunk + 16, lane);
    }
    __syncthreads();
    float* part = total + kWarps * T * 32;
    for (int i = threadIdx.x; i < T * 32; i += kThreads) {
        float v = total[i];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v += total[w * T * 32 + i];
        if (P > 1) {
            part[i] = v;
        } else {
            const int64_t o = static_cast<int64_t>(i >> 5) * H + 32 * chunk + (i & 31);
            if (in_bounds(o < static_cast<int64_t>(T) * H, status)) y[o] = __half_as_ushort(__float2half_rn(v));
        }
    }
    if (P == 1) return;
    cluster_sync_all();
    for (int i = static_cast<int>(threadIdx.x) + rank * kThreads; i < T * 32; i += P * kThreads) {
        const float v = cluster_sum_f1(smem_u32(part + i), P);
        const int64_t o = static_cast<int64_t>(i >> 5) * H + 32 * chunk + (i & 31);
        if (in_bounds(o < static_cast<int64_t>(T) * H, status)) y[o] = __half_as_ushort(__float2half_rn(v));
    }
    cluster_sync_all();
}

template <typename Kern, typename... Args>
cudaError_t launch(Kern kern, dim3 grid, size_t smem, int cluster, cudaStream_t s, Args... args) {
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int NT, bool FP4>
cudaError_t launch_products(const MoeParams& p, const Space& ws, int sm_count, cudaStream_t s, unsigned* status) {
    const int most = p.E < p.T * p.k ? p.E : p.T * p.k;  // experts that can be chosen
    const Matrices up = {static_cast<const uint4*>(p.gate_up_q), p.gate_up_s, p.gate_up_factor, 2 * p.I, p.H, p.G};
    const Matrices down = {static_cast<const uint4*>(p.down_q), p.down_s, p.down_factor, p.H, p.I, p.G};
    const cudaError_t e = launch(gate_up_kernel<NT, FP4>, dim3(static_cast<unsigned>(most * (p.I / 16))), 0, 1, s, up, ws, p.H, p.I, status);
    if (e != cudaSuccess) return e;
    const int chunks = p.H / 32;
    const int64_t steps = most * (padded(p.I) / 128);
    int P = 1;
    while (P < 8 && chunks * P * 2 <= 4 * sm_count && steps / (2 * P * kWarps) >= 2) P *= 2;
    const size_t smem = static_cast<size_t>(kWarps + 1) * p.T * 32 * 4;
    return launch(down_kernel<NT, FP4>, dim3(static_cast<unsigned>(chunks * P)), smem, P, s, down, ws, p.y, p.T, p.H, p.I, P, status);
}

}  // namespace

size_t moe_workspace_bytes(int E, int H, int I) { return space_of(nullptr, E, H, I).bytes; }

cudaError_t launch_moe(const MoeParams& p, int sm_count, cudaStream_t s, unsigned* status) {
    const Space ws = space_of(p.workspace, p.E, p.H, p.I);
    const RouteArgs r = {p.x, p.x_stride, p.router, p.bias, p.ids, p.weights, ws, p.T, p.E, p.H, p.k, p.sigmoid, p.renormalize, p.scale};
    const cudaError_t e = p.T == 1 ? launch(route_kernel<1>, dim3(static_cast<unsigned>(p.E), 1), 0, 1, s, r, status)
                                   : launch(route_kernel<8>, dim3(static_cast<unsigned>(p.E), static_cast<unsigned>((p.T + 7) / 8)), 0, 1, s, r, status);
    if (e != cudaSuccess) return e;
    // Tokens an expert's weights are multiplied by at a time: as many as it has on average when the batch is
    // spread evenly, at least 8; an expert with more reads its weights again.
    const int mean = (p.T * p.k + p.E - 1) / p.E;
    const int nt = p.T <= 8 ? 1 : mean <= 12 ? 2 : 4;
#define W4A16_MOE(NT_) \
    if (nt == NT_) return p.nvfp4 ? launch_products<NT_, true>(p, ws, sm_count, s, status) : launch_products<NT_, false>(p, ws, sm_count, s, status);
    W4A16_MOE(1) W4A16_MOE(2) W4A16_MOE(4)
#undef W4A16_MOE
    return cudaErrorInvalidValue;
}

}  // namespace w4a16
