// A mixture-of-experts layer for a few tokens (T <= 64), its experts' weights in 4 bits:
//
//   l[t][e] = x[t] . router[e]                                     fp16 products, fp32 sums
//   score   = softmax_e(l) or sigmoid(l); chosen: the k experts with the largest l, or score + bias (sigmoid with a bias)
//             (ties: the lower index); r[t][e] = score, over the sum of the chosen ones' if asked, times `scale`
//   a[t][e] = fp16(silu(x[t] . Wg[e]) * (x[t] . Wu[e]))            for the chosen e, products kept in fp32
//   y[t]    = fp16(sum_e r[t][e] * (a[t][e] . Wd[e]))              summed in the order of choice, in fp32
//
// Four kernels on one stream, each scheduled while the one before it runs:
//   route    the logits, a CTA per expert and 8 tokens; the last CTA of 8 tokens chooses their experts, the last of all
//            lists the chosen experts with their tokens
//   gate_up  the listed experts' gate and up columns
//   down     their down columns, r * (a . Wd) of each (token, expert) pair in fp32
//   combine  the sum over a token's k pairs: one order, no atomics
//
// a is rounded to fp16 because it is an operand of the matrix instruction, and as w4a16_silu_mul's is; the gate and up products are
// not. With the rounding of y the layer is off by 2.6e-4 to 3.0e-4 of its size against 64 bits, 2.1e-4 without that of a.
//
// What bounds it is the weights of the chosen experts, read once for every 8, 16 or 32 of an expert's tokens (launch_moe). They go from
// global memory through shared memory into mma.m16n8k16 as the A operand (16 columns of W), tokens are its 8
// columns: a lane (g, t) = (lane / 4, lane % 4) takes the whole 16-byte vector of column g and 32-k block t of
// four adjacent blocks, so that of every 128 k a lane's loads are wide and dense and nothing is exchanged:
// the instruction's k slots are simply numbered so that lane t's are the k of its own block. The B operand
// must follow, so rows of x and of a are kept with their 16-byte units transposed within each 128 (unit w of
// block t at place 4 w + t). A lane copies what it will read itself, so a warp's ring of stages needs no barrier.
//
// Work is a list of items, (listed expert, 32 or 64 columns) over all of K, in steps of 128 k. A CTA takes an equal
// run of items, its warps equal runs of their steps, wherever that cuts an item: the warp that has an item's
// beginning keeps its sums and adds the following warps' parts at the end. All of a warp's steps are one stream of
// copies, whatever items they belong to. The runs are contiguous, so that a CTA meets few experts and finds the
// rows of their tokens in L1.
//
// Measured on one GB300 (hidden 5120, 64 experts of 2176, 8 a token, group 128, in a CUDA graph): 1 token 43 us (139 MB,
// 3.23 TB/s, 0.48 of the measured copy): 9 us of routing, list, starts and ends, then 20 warps an SM that wait for
// their first stages and for one another's items (7.2 items a CTA in gate_up, 8.4 in down: some have 8 and 9). 16 tokens
// 193 us (974 MB, 5.0 TB/s, 0.75; gate_up alone 115 us, 5.7 TB/s): the stream without its products takes 181. 64 tokens
// 272 us (1.1 GB, 4.1 TB/s, 0.60): a step's chain of loads, conversions and products at 3 warps a scheduler, with rows of
// tokens from L2 (all tokens' rows the same one, in L1: 215; without the weights' stream 230); items of 128 columns at 8
// warps, which read the tokens half as often, 284. A cluster of 2 or 4 CTAs with runs of steps in common was slower (46 us
// for one token where one CTA took 41), as were runs cut at any step (48), rows of tokens copied to shared memory with
// the weights (94) and tokens in loads of 32 bytes (43.1 for one, 195 for 16).
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kStages = 2;    // of a warp's ring

// Groups of 16 columns of an item, and warps of a gate_up or down CTA, one CTA an SM, by the tokens (8 NT) that are
// multiplied at a time: as many warps as have the registers for their sums. For 8 tokens, narrow items and many warps:
// one token 42.5 us, 45 with 64 columns and 12 warps, 43.4, 43.7 and 51 with 16, 18 and 22 warps of 32 columns (16 tokens
// 191, 191, 196, 202, 243). For 16, 64 tokens take 272 us, with 32 columns and 12, 16 or 20 warps 307, 279, 424.
__host__ __device__ constexpr int groups_for(int nt) { return nt == 1 ? 2 : 4; }
__host__ __device__ constexpr int warps_for(int nt) { return nt == 1 ? 20 : nt == 2 ? 12 : 8; }

// The weights' formats: how many rows of scales 128 k have.
enum Form {
    kInt4,       // one: groups of a multiple of 128 k
    kInt4Small,  // up to 4: other groups
    kNvfp4       // 8
};

constexpr int kMaxPairs = kMoeMaxTokens * kMoeMaxTop;

// ------------------------------------------------------------------------------------ workspace
// The same layout for every call with the same experts.

// The chosen experts with their tokens. An expert with more than the products take at a time is listed several times,
// each time with the next of them.
struct List {
    int entries;
    uint16_t expert[kMoeMaxExperts + kMaxPairs / 8];
    uint16_t base[kMoeMaxExperts + kMaxPairs / 8 + 1];  // of an entry's first (token, expert) pair
    uint8_t token[kMaxPairs];
    float weight[kMaxPairs];
};

struct Space {
    unsigned* arrived;  // CTAs of each 8 tokens, then the groups
    List* list;
    uint16_t* chosen;   // [tokens][k]
    float* share;       // [tokens][k]
    float* logits;      // [tokens][E]
    int* place;         // [tokens][k]: of a pair in the list
    uint16_t* xp;       // [tokens][Hp], transposed units
    uint16_t* act;      // [pairs][Ip], transposed units
    float* part;        // [pairs][H]
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
    s.list = reinterpret_cast<List*>(take(sizeof(List)));
    s.chosen = reinterpret_cast<uint16_t*>(take(kMaxPairs * 2));
    s.share = reinterpret_cast<float*>(take(kMaxPairs * 4));
    s.logits = reinterpret_cast<float*>(take(static_cast<size_t>(kMoeMaxTokens) * E * 4));
    s.place = reinterpret_cast<int*>(take(kMaxPairs * 4));
    s.xp = reinterpret_cast<uint16_t*>(take(kMoeMaxTokens * padded(H) * 2));
    s.act = reinterpret_cast<uint16_t*>(take(kMaxPairs * padded(I) * 2));
    s.part = reinterpret_cast<float*>(take(static_cast<size_t>(kMaxPairs) * H * 4));
    s.bytes = at;
    return s;
}

// Place of element i of a row with transposed units. Within a unit the pairs lie in the order 0, 2, 1, 3: pairs 0 and 2
// of a word's codes are taken out by one mask, 1 and 3 by another, and each two are the operand of one instruction.
__device__ __forceinline__ int64_t unit_place(int i) {
    return (static_cast<int64_t>(i) & ~127LL) + ((((i >> 3) & 3) * 4 + ((i >> 5) & 3)) << 3) + ((i & 2) << 1) + ((i & 4) >> 1) + (i & 1);
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
    int cap;  // tokens of a list entry
};

// A float as a whole number of the same order, above 1; NaN: 1 (below all).
__device__ __forceinline__ uint32_t order_of(float f) {
    if (f != f) return 1u;
    const uint32_t b = __float_as_uint(f + 0.f);  // -0 and 0 are one value
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// One warp chooses the experts of token t and their weights, of kEach * 32 at most.
template <int kEach>
__device__ __forceinline__ void choose(const RouteArgs& a, int t) {
    const int lane = threadIdx.x & 31;
    uint32_t key[kEach];
    float l[kEach], most = -INFINITY, all = 0.f;
    const float* row = a.w.logits + static_cast<int64_t>(t) * a.E;
#pragma unroll
    for (int i = 0; i < kEach; ++i) l[i] = i * 32 + lane < a.E ? __ldcg(row + i * 32 + lane) : -INFINITY;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int e = i * 32 + lane;
        most = fmaxf(most, l[i]);
        // (without a bias the logits' own order: sigmoids above 17 are all 1 in fp32, below -88 all 0)
        key[i] = e < a.E ? order_of(a.bias ? 1.f / (1.f + expf(-l[i])) + __ldg(a.bias + e) : l[i]) : 0u;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (!a.sigmoid && !a.renormalize) {
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (i * 32 + lane < a.E) all += expf(l[i] - most);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    int mine = 0;
    float value = 0.f;  // of the expert in place `lane`
    for (int r = 0; r < a.k; ++r) {  // the largest left
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < kEach; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(0xffffffffu, best);
        uint32_t at = 0xFFFFFFFFu;
        float v = 0.f;
#pragma unroll
        for (int i = kEach - 1; i >= 0; --i)
            if (key[i] == best) {
                at = static_cast<uint32_t>(i * 32 + lane);
                v = l[i];
            }
        at = __reduce_min_sync(0xffffffffu, at);
        v = __shfl_sync(0xffffffffu, v, at & 31u);
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (static_cast<uint32_t>(i * 32 + lane) == at) key[i] = 0;
        if (lane == r) {
            mine = static_cast<int>(at);
            value = v;
        }
    }
    float s = lane < a.k ? (a.sigmoid ? 1.f / (1.f + expf(-value)) : expf(value - most)) : 0.f;
    if (a.renormalize) {
        if (a.sigmoid) {  // far below 0 a sigmoid is e^l, and its share is the same relative to the largest chosen: no sum of tiny numbers
            float top = lane < a.k ? value : -INFINITY;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (top < -20.f && top > -INFINITY) s = lane < a.k ? expf(value - top) : 0.f;  // (1 + e^l is 1 in fp32)
        }
        all = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    if (a.renormalize || !a.sigmoid) s = all == 0.f ? 0.f : __fdiv_rn(s, all);  // (sigmoids of -inf are 0; a NaN goes on to all)
    if (lane < a.k) {
        const int p = t * a.k + lane;
        a.w.chosen[p] = static_cast<uint16_t>(mine);
        a.w.share[p] = s * a.scale;
        if (a.ids) a.ids[p] = mine;
        if (a.weights) a.weights[p] = s * a.scale;
    }
    if (a.T == 1) {  // the list at once: an entry a lane
        int at = 0;
        for (int o = 0; o < a.k; ++o) at += __shfl_sync(0xffffffffu, mine, o) < mine;
        if (lane < a.k) {
            List& list = *a.w.list;
            list.expert[at] = static_cast<uint16_t>(mine);
            list.base[at] = static_cast<uint16_t>(at);
            list.token[at] = 0;
            list.weight[at] = s * a.scale;
            a.w.place[lane] = at;
            if (lane == 0) list.entries = a.k;
        }
    }
}

// The list, made by one CTA.
__device__ __forceinline__ void make_list(const RouteArgs& a, unsigned* status) {
    constexpr int kW = kRouteThreads / 32;
    __shared__ uint32_t mask[2][kMoeMaxExperts];  // tokens of an expert, one bit each
    __shared__ uint16_t start[kMoeMaxExperts];    // of its pairs
    __shared__ uint32_t sums[kW];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, pairs = a.T * a.k;
    List& list = *a.w.list;
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) mask[0][e] = mask[1][e] = 0;
    __syncthreads();
    // Read once: that every token's bit is set in its expert's mask is what keeps the places below within the list, also
    // where another call on the same workspace changes `chosen` meanwhile (which is not allowed, and gives wrong results only).
    int expert[kMaxPairs / kRouteThreads];
#pragma unroll
    for (int i = 0; i < kMaxPairs / kRouteThreads; ++i) {
        const int p = i * kRouteThreads + static_cast<int>(threadIdx.x), t = p / a.k;
        if (p >= pairs) continue;
        expert[i] = min(static_cast<int>(__ldcg(a.w.chosen + p)), a.E - 1);
        atomicOr(&mask[t >> 5][expert[i]], 1u << (t & 31));
    }
    uint32_t carry = 0;  // (entries << 16) + pairs of the experts before
    for (int e0 = 0; e0 < a.E; e0 += kRouteThreads) {
        __syncthreads();
        const int e = e0 + static_cast<int>(threadIdx.x);
        const uint32_t n = e < a.E ? __popc(mask[0][e]) + __popc(mask[1][e]) : 0u, own = ((n + a.cap - 1) / a.cap << 16) + n;
        uint32_t upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) sums[warp] = upto;
        __syncthreads();
        upto += carry;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            if (w < warp) upto += sums[w];
            carry += sums[w];
        }
        const uint32_t before = upto - own;
        int at = static_cast<int>(before >> 16);
        for (uint32_t i = 0; i < n; i += a.cap) {
            list.expert[at] = static_cast<uint16_t>(e);
            list.base[at++] = static_cast<uint16_t>((before & 0xFFFFu) + i);
        }
        if (e < a.E) start[e] = static_cast<uint16_t>(before & 0xFFFFu);
    }
    if (threadIdx.x == 0) {
        list.entries = static_cast<int>(carry >> 16);
        list.base[carry >> 16] = static_cast<uint16_t>(carry & 0xFFFFu);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMaxPairs / kRouteThreads; ++i) {  // an expert's pairs by token
        const int p = i * kRouteThreads + static_cast<int>(threadIdx.x), t = p / a.k, e = expert[i];
        if (p >= pairs) continue;
        const uint32_t lo = mask[0][e], hi = mask[1][e], bit = 1u << (t & 31);
        const int at = start[e] + (t < 32 ? __popc(lo & (bit - 1)) : __popc(lo) + __popc(hi & (bit - 1)));
        if (!in_bounds(at < pairs, status)) continue;
        list.token[at] = static_cast<uint8_t>(t);
        list.weight[at] = __ldcg(a.w.share + p);
        a.w.place[p] = at;
    }
}

// Whether this CTA is the last of `of` that arrive at `counter`, which is then ready for the next call.
__device__ __forceinline__ bool last_of(unsigned* counter, unsigned of) {
    __shared__ int last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(counter, 1u) == of - 1u;
        if (last) *counter = 0;
        __threadfence();
    }
    __syncthreads();
    return last != 0;
}

// TB tokens a CTA (1 or 8), one expert.
template <int TB>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteArgs a, unsigned* status) {
    constexpr int kW = kRouteThreads / 32;
    __shared__ float part[kW][TB];
    griddep_launch_dependents();
    const int e = blockIdx.x, t0 = blockIdx.y * TB;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tokens = min(TB, a.T - t0), vecs = a.H / 8;
    const uint16_t* wrow = a.router + static_cast<int64_t>(e) * a.H;
    griddep_wait();  // before any load: the router may be an earlier kernel's output as well
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (static_cast<int>(threadIdx.x) < vecs) w = *reinterpret_cast<const uint4*>(wrow + 8 * threadIdx.x);
    float acc[TB][2];
#pragma unroll
    for (int i = 0; i < TB; ++i) acc[i][0] = acc[i][1] = 0.f;
    for (int v = threadIdx.x; v < vecs; v += kRouteThreads) {
        uint4 x[TB];
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            const int64_t at = (t0 + i) * a.x_stride + 8 * static_cast<int64_t>(v);
            x[i] = i < tokens && in_bounds(8 * v + 8 <= a.H, status) ? *reinterpret_cast<const uint4*>(a.x + at) : make_uint4(0u, 0u, 0u, 0u);
        }
        const int next = v + kRouteThreads;
        const uint4 wn = next < vecs ? *reinterpret_cast<const uint4*>(wrow + 8 * next) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            fma2_mixed(acc[i][0], acc[i][1], w.x, x[i].x);
            fma2_mixed(acc[i][0], acc[i][1], w.y, x[i].y);
            fma2_mixed(acc[i][0], acc[i][1], w.z, x[i].z);
            fma2_mixed(acc[i][0], acc[i][1], w.w, x[i].w);
        }
        w = wn;
    }
    for (int i = e; i < tokens; i += a.E)  // a token's row as the products want it
        for (int v = threadIdx.x; v < vecs; v += kRouteThreads) {
            const uint4 q = *reinterpret_cast<const uint4*>(a.x + (t0 + i) * a.x_stride + 8 * static_cast<int64_t>(v));
            *reinterpret_cast<uint4*>(a.w.xp + padded(a.H) * (t0 + i) + unit_place(8 * v)) = make_uint4(q.x, q.z, q.y, q.w);
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
        for (int i = 1; i < kW; ++i) s += part[i][threadIdx.x];
        a.w.logits[static_cast<int64_t>(t0 + threadIdx.x) * a.E + e] = s;
    }
    if (!last_of(a.w.arrived + blockIdx.y, gridDim.x)) return;
    if (warp < tokens) {
        if (a.E <= 64)
            choose<2>(a, t0 + warp);
        else if (a.E <= 256)
            choose<8>(a, t0 + warp);
        else
            choose<kMoeMaxExperts / 32>(a, t0 + warp);
    }
    if (TB == 1) return;
    if (gridDim.y > 1 && !last_of(a.w.arrived + 15, gridDim.y)) return;
    __syncthreads();
    make_list(a, status);
}

// ------------------------------------------------------------------------------------ products
struct Matrices {
    const uint4* w;       // repacked codes of all experts
    const uint16_t* s;    // repacked scales
    const float* factor;  // NVFP4: fp32 scale of each expert's matrix
    int N, K, G;          // of one expert
    int E;
};

// D (16 columns x 8 tokens) += A (16 columns x 16 k) . B (16 k x 8 tokens)
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A stage of a warp's ring: 128 k of C * 16 columns. Vectors: [16 columns][half][32-k block][column, swizzled]; then scales
// [row][columns]. Column g of block t lies at place g ^ 2 t of its 8, so that neither the copies (8 columns of
// a block at a time) nor the reads (2 columns of 4 blocks) meet in a bank.
template <Form F, int C>
struct Stage {
    static constexpr int kRows = F == kInt4 ? 1 : F == kInt4Small ? 4 : 8;  // of scales
    static constexpr int kScales = 1024 * C;
    static constexpr int kBytes = kScales + kRows * 32 * C;
};
__device__ __forceinline__ uint32_t vector_place(int lane) {
    const int g = lane >> 2, t = lane & 3;
    return static_cast<uint32_t>(t * 128 + ((g ^ (2 * t)) & 7) * 16);
}

// Where a lane's copies come from: an item's columns, at the next step to be copied. A block's vectors lie side by side.
template <Form F, int C>
struct Source {
    const uint4* w;
    const uint16_t* s;  // kInt4: of this lane's pair (of 32 columns: of the first 16 lanes')
    int wt;             // vectors from one 32-k block to the next
    int kb, row_left;   // kInt4: steps until the next row of scales

    static __device__ __forceinline__ int pair_of(int lane) { return 2 * (lane % (8 * C)); }
    __device__ __forceinline__ void set(const Matrices& m, int expert, int column, int first, int lane) {
        const int blocks = m.K / 32, rows = m.K / m.G, tile = column >> 7;
        kb = first;
        wt = min(128, m.N - 128 * tile);
        w = m.w + static_cast<int64_t>(expert) * m.N * blocks + static_cast<int64_t>(tile) * 128 * blocks + (column & 127) + (lane >> 2) +
            static_cast<int64_t>(4 * first + (lane & 3)) * wt;
        s = m.s + static_cast<int64_t>(expert) * m.N * rows + static_cast<int64_t>(tile) * 128 * rows + (column & 127);
        if (F == kInt4) {
            const int q = m.G / 128, row = first / q;
            s += static_cast<int64_t>(row) * wt + pair_of(lane);
            row_left = q - (first - row * q);
        }
    }
    // per: 32-k blocks a scale row, shift its logarithm or -1
    __device__ __forceinline__ void copy(const Matrices& m, uint32_t stage, int blocks, int per, int shift, int lane, unsigned* status) {
        const uint32_t vec = stage + vector_place(lane);
        const int64_t all = static_cast<int64_t>(m.E) * m.N, scales = all * (m.K / m.G);  // (index checks)
        if ((F == kInt4 || kb * 4 + (lane & 3) < blocks) && in_bounds(w - m.w + 16 * C - 8 < all * blocks, status)) {
#pragma unroll
            for (int i = 0; i < 2 * C; ++i) copy16(vec + 512u * i, w + 8 * i);
        }
        w += 4 * wt;
        const uint32_t to = stage + Stage<F, C>::kScales + 2u * pair_of(lane);
        const bool one = 2 * lane < 16 * C;  // of the lanes that copy scales
        if (F == kInt4) {
            if (one && in_bounds(s - m.s + 2 <= scales, status)) copy4(to, s);
            if (--row_left == 0) {
                row_left = per >> 2;
                s += wt;
            }
        } else {
#pragma unroll
            for (int r = 0; r < Stage<F, C>::kRows; ++r) {
                const int blk = F == kNvfp4 ? kb * 4 + (r >> 1) : kb * 4 + r;
                if (blk >= blocks) continue;
                const int row = F == kNvfp4 ? kb * 8 + r : shift >= 0 ? blk >> shift : blk / per;
                const uint16_t* q = s + static_cast<int64_t>(row) * wt + pair_of(lane);
                if (one && in_bounds(q - m.s + 2 <= scales, status)) copy4(to + 32u * C * r, q);
            }
        }
        ++kb;
    }
};

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int w) { return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w; }

// A lane's tokens, one of each 8: where its row has the step's units, and what was read there.
template <int NT>
struct Tokens {
    uint32_t row[NT];  // (below 2^32: 1024 rows of 65,536 at most)
    uint4 unit[NT][4];
};

// sum[c][n] += 16 columns c of a stage times 8 tokens n, TILES * 8 tokens. The units of the next step, `on` elements on,
// are asked for as soon as this step's are done with (`ahead`: there is one of the same tokens).
//
// FAST (int4): the pairs of codes that a mask takes out of a word are, as fp16 numbers, q 2^-24 (bits 0..3) or q 2^-20
// (bits 4..7): subnormal and exact. One fused multiply-add with s 2^20 and -s / 2 or -8 s gives (q - 8) s / 16 or
// (q - 8) s with its one rounding, which is the format's: 9 instructions for 8 weights instead of dequant8's 13. It needs
// every number normal, a scale in 2^-10 .. 2^-4; other steps go the long way (all of them: one token 45.4 us instead of 42.5,
// 64 tokens 292 instead of 272; without the question 41.7 and 276). Sixteenths are summed apart, or, where there are registers for one set of sums only,
// codes are multiplied by 16 first, 11 instructions (one token 43.7 us that way, 16 tokens 199; 64 tokens 304 apart).
__host__ __device__ constexpr bool apart(int nt) { return nt == 1; }

template <int NT, int TILES, Form F, bool FAST, int C = groups_for(NT)>
__device__ __forceinline__ void multiply(float (&sum)[C][NT][4], float (&sixteenth)[C][NT][4], uint32_t stage, Tokens<NT>& x,
                                         const uint16_t* rows, int on, bool ahead, bool there, int lane) {
    constexpr bool kApart = apart(NT);
    constexpr uint32_t k16 = 0x4C004C00u;  // (16, 16)
    const uint32_t vec = stage + vector_place(lane), sc = stage + Stage<F, C>::kScales + 2u * (lane >> 2);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const uint4 v[2] = {lds128(vec + 1024u * c), lds128(vec + 1024u * c + 512u)};
        uint32_t s[2][2];  // of columns g, g + 8, twice in a register; NVFP4: of a block's halves
        const uint32_t row = F == kInt4 ? 0u : F == kInt4Small ? lane & 3u : 2u * (lane & 3u);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            s[i][0] = lds16(sc + 32u * C * row + 32u * c + 16u * i) * 0x10001u;
            if (F == kNvfp4) s[i][1] = lds16(sc + 32u * C * (row + 1) + 32u * c + 16u * i) * 0x10001u;
            if (F != kInt4 && !there) s[i][0] = s[i][1] = 0x1C001C00u;  // past K: what the stage holds is not of this step
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t d[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t word = word_of(v[i], w);
                if (F == kNvfp4) {
                    dequant8_nvfp4(word, s[i][w >> 1], d[i]);
                } else if (!FAST) {
                    dequant8(word, s[i][0], d[i]);
                } else {
                    const uint32_t up = s[i][0] + 0x50005000u, less_half = s[i][0] + 0x7C007C00u, less_8 = s[i][0] + 0x8C008C00u;
                    d[i][0] = kApart ? hfma2(word & 0x000F000Fu, up, less_half) : hfma2(hmul2(word & 0x000F000Fu, k16), up, less_8);
                    d[i][1] = hfma2(word & 0x00F000F0u, up, less_8);
                    d[i][2] = kApart ? hfma2((word >> 8) & 0x000F000Fu, up, less_half) : hfma2(hmul2((word >> 8) & 0x000F000Fu, k16), up, less_8);
                    d[i][3] = hfma2((word >> 8) & 0x00F000F0u, up, less_8);
                }
            }
#pragma unroll
            for (int n = 0; n < TILES; ++n) {
                if (F != kInt4 && c == 0 && !there) x.unit[n][w] = make_uint4(0u, 0u, 0u, 0u);
                const uint4& u = x.unit[n][w];
                mma16816(FAST && kApart ? sixteenth[c][n] : sum[c][n], d[0][0], d[1][0], d[0][2], d[1][2], u.x, u.y);
                mma16816(sum[c][n], d[0][1], d[1][1], d[0][3], d[1][3], u.z, u.w);
                if (c == C - 1 && ahead) x.unit[n][w] = *reinterpret_cast<const uint4*>(rows + x.row[n] + on + 32 * w);
            }
        }
    }
}

// Whether all scales of a step are normal enough for the fast way: 2^-10 <= s < 2^-4. (A row past K is not looked at.)
template <Form F, int C>
__device__ __forceinline__ bool scales_fit(uint32_t stage, int kb, int blocks, int lane) {
    bool fit = true;
#pragma unroll
    for (int r = 0; r < Stage<F, C>::kRows; ++r) {
        if (F != kInt4 && kb * 4 + r >= blocks) continue;
        const uint32_t p = lds32(stage + Stage<F, C>::kScales + 32u * C * r + 4u * (lane % (8 * C)));
        fit = fit && (p & 0xFFFFu) - 0x1400u < 0x1800u && (p >> 16) - 0x1400u < 0x1800u;
    }
    return __all_sync(0xffffffffu, fit);
}

// DOWN false: gate and up (16 columns of gate, the 16 of up, twice an item), true: down.
template <int NT, Form F, bool DOWN>
__global__ void __launch_bounds__(warps_for(NT) * 32, 1) experts_kernel(const Matrices m, const RouteArgs r, int I, unsigned* status) {
    constexpr int kWarps = warps_for(NT), C = groups_for(NT);
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ List list;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, H = r.H;
    const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(warp * kStages * Stage<F, C>::kBytes);
    // parts of items that begin in an earlier warp: [warp][16 columns][8 tokens][register][lane]
    float* heads = reinterpret_cast<float*>(smem + kWarps * kStages * Stage<F, C>::kBytes);
    if (!DOWN) {
        griddep_wait();
        griddep_launch_dependents();  // (after the wait: the next kernel may read the list before its own)
    } else {
        griddep_launch_dependents();
        // The list is the work of the kernel before the last: complete, since every CTA of the last one had passed its
        // wait before this kernel could start.
    }
    {  // Every number within its limits: a workspace that was not zeroed, or that two calls
       // share, gives wrong results only (one token 0.7 us more, 16 tokens 2).
        const List* from = r.w.list;
        const int pairs = r.T * r.k, most = min(pairs, kMoeMaxExperts + kMaxPairs / 8);  // (no more entries than pairs)
        const int entries = max(1, min(__ldcg(&from->entries), most));
        for (int i = threadIdx.x; i < most; i += kWarps * 32) {
            list.expert[i] = static_cast<uint16_t>(min(static_cast<int>(__ldcg(from->expert + i)), m.E - 1));
            list.base[i] = static_cast<uint16_t>(min(static_cast<int>(__ldcg(from->base + i)), pairs - 1));
        }
        for (int i = threadIdx.x; i < pairs; i += kWarps * 32) {
            if (DOWN)
                list.weight[i] = __ldcg(from->weight + i);
            else
                list.token[i] = static_cast<uint8_t>(min(static_cast<int>(__ldcg(from->token + i)), r.T - 1));
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            list.entries = entries;
            list.base[entries] = static_cast<uint16_t>(pairs);
        }
        __syncthreads();
    }

    const int chunks = m.N / (16 * C);
    const int steps = static_cast<int>(padded(m.K) / 128), blocks = m.K / 32;
    const int per = F == kNvfp4 ? 1 : m.G / 32, shift = (per & (per - 1)) == 0 ? __ffs(per) - 1 : -1;
    const int64_t items = static_cast<int64_t>(list.entries) * chunks;
    const int64_t item0 = items * blockIdx.x / gridDim.x;
    const int run = static_cast<int>(items * (blockIdx.x + 1) / gridDim.x - item0) * steps;  // this CTA's steps
    auto begin = [&](int w) { return static_cast<int>(static_cast<int64_t>(run) * w / kWarps); };
    const int s0 = begin(warp), s1 = begin(warp + 1);

    // the copying end of the stream
    Source<F, C> src;
    const int64_t first = item0 + s0 / steps;
    int entry = static_cast<int>(first / chunks), chunk = static_cast<int>(first % chunks), kb = s0 % steps;
    int c_entry = entry, c_chunk = chunk, c_left = s1 - s0;
    auto fetch = [&](int slot) {
        if (c_left > 0) {
            src.copy(m, ring + static_cast<uint32_t>(slot * Stage<F, C>::kBytes), blocks, per, shift, lane, status);
            if (--c_left > 0 && src.kb == steps) {
                if (++c_chunk == chunks) {
                    c_chunk = 0;
                    ++c_entry;
                }
                src.set(m, list.expert[c_entry], 16 * C * c_chunk, 0, lane);
            }
        }
        copies_commit();
    };
    if (c_left > 0) src.set(m, list.expert[c_entry], 16 * C * c_chunk, kb, lane);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    if (DOWN) griddep_wait();

    const uint16_t* const rows_of = DOWN ? r.w.act : r.w.xp;
    Tokens<NT> x;  // at step kb
    float acc[C][NT][4], sixteenth[C][NT][4];
    constexpr bool kFast = F != kNvfp4;
    int base = 0, count = 0, tiles = 1;
    const int width = static_cast<int>(padded(m.K));
    auto meet = [&]() {  // the rows of an entry's tokens at step kb; a place without a token reads the first one's
        base = list.base[entry];
        count = list.base[entry + 1] - base;
        tiles = (count + 7) / 8;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int i = 8 * n + (lane >> 2), pair = base + (i < count ? i : 0);
            int row = DOWN ? pair : list.token[pair];
            if (!in_bounds(row >= 0 && row < (DOWN ? r.T * r.k : r.T), status)) row = 0;
            x.row[n] = static_cast<uint32_t>(row * width + kb * 128 + (lane & 3) * 8);
            if (n > 0 && n >= tiles) continue;
#pragma unroll
            for (int w = 0; w < 4; ++w) x.unit[n][w] = *reinterpret_cast<const uint4*>(rows_of + x.row[n] + 32 * w);
        }
    };
    auto clear = [&]() {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[c][n][i] = sixteenth[c][n][i] = 0.f;
    };
    auto fold = [&]() {
        if constexpr (kFast && apart(NT)) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[c][n][i] = fmaf(16.f, sixteenth[c][n][i], acc[c][n][i]);
        }
    };
    auto finish = [&]() {  // a lane's columns g, g + 8 of each 16 for tokens 2 t, 2 t + 1 of 8
        const float factor = F == kNvfp4 ? m.factor[list.expert[entry]] : 1.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (n > 0 && n >= tiles) break;
                const int i = 8 * n + 2 * (lane & 3) + h, pair = base + i;
                const bool there = i < count && in_bounds(i >= count || pair < kMaxPairs, status);
                if (DOWN) {
                    if (!there) continue;
                    const float w = list.weight[pair] * factor;
                    float* to = r.w.part + static_cast<int64_t>(pair) * H + 16 * C * chunk + (lane >> 2);
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        to[16 * c] = w * acc[c][n][h];
                        to[16 * c + 8] = w * acc[c][n][2 + h];
                    }
                } else {
                    if (!there) continue;
#pragma unroll
                    for (int q = 0; q < C; ++q) {
                        const float g = acc[q & ~1][n][2 * (q & 1) + h] * factor, u = acc[(q & ~1) + 1][n][2 * (q & 1) + h] * factor;
                        r.w.act[pair * padded(I) + unit_place(8 * C * chunk + 8 * q + (lane >> 2))] =
                            __half_as_ushort(__float2half_rn(g / (1.0f + expf(-g)) * u));
                    }
                }
            }
    };
    float* mine = heads + (warp * C * NT * 4) * 32 + lane;
    auto leave = [&]() {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) mine[((c * NT + n) * 4 + i) * 32] = acc[c][n][i];
    };

    bool whole = kb == 0;  // the item's beginning is this warp's
    clear();
    if (s0 < s1) meet();
    int slot = 0;
    for (int s = s0; s < s1; ++s) {
        copies_wait<kStages - 2>();
        __syncwarp();  // (scales are copied for each other; and the slot that is filled next has been read)
        fetch(slot == 0 ? kStages - 1 : slot - 1);
        const uint32_t stage = ring + static_cast<uint32_t>(slot * Stage<F, C>::kBytes);
        const bool there = F == kInt4 || kb * 4 + (lane & 3) < blocks;
        const bool last = kb + 1 == steps, ahead = s + 1 < s1 && !(last && chunk + 1 == chunks);
        const int on = last ? 128 - width : 128;  // the next item's first step, of the same tokens
        auto go = [&](auto fast) {
            constexpr bool kGo = decltype(fast)::value;
            if (NT == 1 || tiles == 1)
                multiply<NT, 1, F, kGo>(acc, sixteenth, stage, x, rows_of, on, ahead, there, lane);
            else if (NT == 2 || tiles == 2)
                multiply<NT, NT < 2 ? 1 : 2, F, kGo>(acc, sixteenth, stage, x, rows_of, on, ahead, there, lane);
            else
                multiply<NT, NT, F, kGo>(acc, sixteenth, stage, x, rows_of, on, ahead, there, lane);
        };
        if (kFast && scales_fit<F, C>(stage, kb, blocks, lane))
            go(std::integral_constant<bool, kFast>());
        else
            go(std::false_type());
        if (++slot == kStages) slot = 0;
#pragma unroll
        for (int n = 0; n < NT; ++n) x.row[n] += static_cast<uint32_t>(on);
        if (++kb == steps) {
            fold();
            if (whole)
                finish();
            else
                leave();
            clear();
            whole = true;
            kb = 0;
            if (++chunk == chunks) {
                chunk = 0;
                ++entry;
                if (s + 1 < s1) meet();
            }
        }
    }
    copies_wait<0>();
    const bool open = s0 < s1 && kb != 0;
    if (open) fold();
    if (open && !whole) leave();
    __syncthreads();
    if (open && whole) {
        const int end = s1 - kb + steps;  // of the item, in the CTA's steps
        constexpr int kBatch = NT == 2 ? 2 : 1, kValues = 4 * C * NT;
        for (int other = warp + 1; other < kWarps && begin(other) < end; other += kBatch) {
            float v[kBatch][kValues];
#pragma unroll
            for (int o = 0; o < kBatch; ++o) {
                const int w = other + o;
                const bool part = w < kWarps && begin(w) < end && begin(w) < begin(w + 1);
                const float* from = heads + w * kValues * 32 + lane;
#pragma unroll
                for (int i = 0; i < kValues; ++i)
                    v[o][i] = part ? from[32 * i] : 0.f;
            }
#pragma unroll
            for (int o = 0; o < kBatch; ++o)
#pragma unroll
                for (int i = 0; i < kValues; ++i) acc[i / (4 * NT)][i / 4 % NT][i % 4] += v[o][i];
        }
        finish();
    }
}

// y of a token: its pairs' sums in the order of choice. Four columns a thread.
__global__ void __launch_bounds__(256) combine_kernel(const Space ws, uint16_t* __restrict__ y, int T, int H, int k, unsigned* status) {
    griddep_launch_dependents();
    const int64_t i = blockIdx.x * 256LL + threadIdx.x;
    const int quads = H / 4;
    const int t = static_cast<int>(i / quads), c = static_cast<int>(i % quads) * 4;
    const bool there = t < T;
    // (the places are route's work: complete before down could start, and so before this kernel could)
    int pair[kMoeMaxTop];
#pragma unroll
    for (int j = 0; j < kMoeMaxTop; ++j) pair[j] = there && j < k ? max(0, min(__ldcg(ws.place + t * k + j), T * k - 1)) : 0;
    griddep_wait();
    if (!there) return;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j0 = 0; j0 < kMoeMaxTop; j0 += 8) {
        if (j0 >= k) break;
        float4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = j0 + j < k && in_bounds(pair[j0 + j] >= 0 && pair[j0 + j] < T * k, status)
                       ? __ldcg(reinterpret_cast<const float4*>(ws.part + static_cast<int64_t>(pair[j0 + j]) * H + c))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sum.x += v[j].x;
            sum.y += v[j].y;
            sum.z += v[j].z;
            sum.w += v[j].w;
        }
    }
    const __half2 lo = __floats2half2_rn(sum.x, sum.y), hi = __floats2half2_rn(sum.z, sum.w);
    *reinterpret_cast<uint2*>(y + static_cast<int64_t>(t) * H + c) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

template <typename Kern, typename... Args>
cudaError_t launch(Kern kern, dim3 grid, int threads, size_t smem, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int NT, Form F>
cudaError_t launch_form(const MoeParams& p, const RouteArgs& r, int sm_count, cudaStream_t s, unsigned* status) {
    const Matrices up = {static_cast<const uint4*>(p.gate_up_q), p.gate_up_s, p.gate_up_factor, 2 * p.I, p.H, p.G, p.E};
    const Matrices down = {static_cast<const uint4*>(p.down_q), p.down_s, p.down_factor, p.H, p.I, p.G, p.E};
    constexpr int kThreads = warps_for(NT) * 32;
    constexpr int C = groups_for(NT);
    constexpr size_t smem = warps_for(NT) * (kStages * Stage<F, C>::kBytes + C * NT * 4 * 32 * 4);
    const dim3 grid(static_cast<unsigned>(sm_count));
    static std::atomic<uint64_t> allowed{0};  // devices that know these kernels' shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || (allowed.load() >> dev & 1) == 0) {
        e = cudaFuncSetAttribute(experts_kernel<NT, F, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(experts_kernel<NT, F, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        if (dev < 64) allowed.fetch_or(uint64_t{1} << dev);
    }
    e = launch(experts_kernel<NT, F, false>, grid, kThreads, smem, s, up, r, p.I, status);
    if (e != cudaSuccess) return e;
    return launch(experts_kernel<NT, F, true>, grid, kThreads, smem, s, down, r, p.I, status);
}

template <int NT>
cudaError_t launch_products(const MoeParams& p, const RouteArgs& r, int sm_count, cudaStream_t s, unsigned* status) {
    if (p.nvfp4) return launch_form<NT, kNvfp4>(p, r, sm_count, s, status);
    return p.G % 128 == 0 ? launch_form<NT, kInt4>(p, r, sm_count, s, status) : launch_form<NT, kInt4Small>(p, r, sm_count, s, status);
}

}  // namespace

size_t moe_workspace_bytes(int E, int H, int I) { return space_of(nullptr, E, H, I).bytes; }

cudaError_t launch_moe(const MoeParams& p, int sm_count, cudaStream_t s, unsigned* status) {
    const Space ws = space_of(p.workspace, p.E, p.H, p.I);
    // Tokens that an expert's weights are multiplied by at a time: 8 where the average expert has few (the kernel with
    // the most warps), 16, or 32; an expert with more is streamed again.
    const int nt = p.T <= 8 || p.T * p.k <= 3 * p.E ? 1 : p.T * p.k <= 10 * p.E || p.T <= 16 ? 2 : 4;
    const RouteArgs r = {p.x, p.x_stride, p.router, p.bias, p.ids, p.weights, ws, p.T, p.E, p.H, p.k, p.sigmoid, p.renormalize, p.scale, 8 * nt};
    cudaError_t e = p.T == 1 ? launch(route_kernel<1>, dim3(static_cast<unsigned>(p.E), 1), kRouteThreads, 0, s, r, status)
                             : launch(route_kernel<8>, dim3(static_cast<unsigned>(p.E), static_cast<unsigned>((p.T + 7) / 8)), kRouteThreads, 0, s, r, status);
    if (e != cudaSuccess) return e;
    e = nt == 1 ? launch_products<1>(p, r, sm_count, s, status)
        : nt == 2 ? launch_products<2>(p, r, sm_count, s, status)
                  : launch_products<4>(p, r, sm_count, s, status);
    if (e != cudaSuccess) return e;
    return launch(combine_kernel, dim3(static_cast<unsigned>((static_cast<int64_t>(p.T) * p.H / 4 + 255) / 256)), 256, 0, s, ws, p.y, p.T, p.H, p.k, status);
}

}  // namespace w4a16
