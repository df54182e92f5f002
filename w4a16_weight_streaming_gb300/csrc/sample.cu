// Token sampling: temperature, top-k, top-p and min-p from a given uniform number per row, without a sort.
//
//   order   logits descending, ties by lower index (NaN and -inf: masked, never chosen)
//   weight  W = rne(2^40 w), w = exp((l - l_max) / T) in binary32, w = 1 where l = l_max
//   kept    the first k; of those, each whose preceding mass is below p times their mass; w >= min_p;
//           the first one always
//   token   the first kept one at which the running mass exceeds u times the kept mass
//
// Weights are whole numbers, so every mass is an exact 64-bit sum: the result does not depend on the
// order of additions, and repeats are identical. Two kernels:
//
// Every kept set is the beginning of one order, so a cut is known by the mass before it, and the smallest
// of the cuts' masses is the kept mass; the draw is a position in the same running mass. fp16 logits have
// at most 65,536 values and equal logits have equal weights, so a row is described by how often each value
// occurs, and its weight is computed once a value.
//
// Window: the first kernel counts the 4096 values below the largest logit (4 octaves), one shared-memory
// atomic each, after a first pass that finds the largest. Where the mass of all tokens is asked for, the
// weights of those below the window are added up directly. A row is one CTA or a thread-block cluster
// whose counts are added up in rank 0. Draws and cuts below the window are left to the second kernel.
//
// Counting, for the rest: a cluster per row counts all its values in shared memory (16-bit counters, each
// CTA's slice is below 65,536 elements). Each CTA then adds up the cluster's counts of its share of the
// values and folds them into coarse bins of 32 values, count and mass. Every decision is a search in the
// 2048 prefix sums followed by a look at the 32 values of one bin.
//
// Measured on one GB300, vocabulary 248,320: 1 row with top-k 20 and top-p 12.1 us, 16 rows with min-p 12.0 us:
// latency, of two short passes and the barriers behind them. 256 rows with top-p alone 112 us (127 MB, 1.13 TB/s):
// the issue of some 40 instructions a logit, most of them for the exponentials of those below the window and
// the counts. 33 rows of 32,003 with settings of their own 22.5 us: rank 0's weights and decisions.
#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 512;
constexpr int kBins = 2048;           // coarse bins of 32 adjacent values
constexpr uint32_t kMaskedKey = 0x03FFu;  // -inf; every finite value's key is above
constexpr size_t kHistBytes = 65536 * 2;
constexpr size_t kSmemBytes = kHistBytes + 1024 + kBins * (8 + 4) + 65536;  // + the summed counts, C >= 4

// fp16 bits -> a 16-bit key in the order of the numbers (-0 and +0 share one); masked values <= kMaskedKey.
__device__ __forceinline__ uint32_t key_of(uint32_t bits) {
    if ((bits & 0x7FFFu) > 0x7C00u) return kMaskedKey;  // NaN
    if (bits == 0x8000u) bits = 0;
    return (bits & 0x8000u) ? (~bits & 0xFFFFu) : (bits | 0x8000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    const uint32_t bits = (key & 0x8000u) ? (key & 0x7FFFu) : (~key & 0xFFFFu);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}

struct Softmax {
    uint32_t kmax;
    float vmax, temp;
    __device__ __forceinline__ float weight(uint32_t key) const {
        return key == kmax ? 1.f : expf(__fdiv_rn(__fsub_rn(value_of(key), vmax), temp));
    }
    __device__ __forceinline__ unsigned long long fixed(uint32_t key) const {
        return __float2ull_rn(weight(key) * 1099511627776.f);  // 2^40, exact
    }
};

// The smallest key with weight >= w (0 < w <= 1), found by every lane of a warp: 32 keys at a time.
__device__ __forceinline__ uint32_t smallest_key(const Softmax& sm, float w) {
    const int lane = threadIdx.x & 31;
    uint32_t base = 0, width = 65536;
    while (width > 1) {
        const uint32_t step = max(1u, width / 32);
        const uint32_t key = min(base + (lane + 1) * step - 1, sm.kmax);
        const bool yes = key > kMaskedKey && sm.weight(key) >= w;
        base += (__ffs(__ballot_sync(0xffffffffu, yes)) - 1) * step;
        width = step;
    }
    return base;
}

// floor(total * n24 / 2^24) in 64-bit whole numbers, total < 2^60, n24 <= 2^24
__device__ __forceinline__ unsigned long long scaled(unsigned long long total, unsigned long long n24) {
    return n24 * (total >> 24) + ((n24 * (total & 0xFFFFFFull)) >> 24);
}

__device__ __forceinline__ uint32_t ld_dsmem_u16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared::cluster.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint4 ld_dsmem_u4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void st_dsmem_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_dsmem_u4(uint32_t addr, const uint4& v) {
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void st_dsmem_u64(uint32_t addr, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// What the last element of a bin's search knows about the values of one bin, one value a lane, in
// descending order: the whole cluster's count of the value, and what precedes it.
struct Fine {
    uint32_t key, count, count_before;
    unsigned long long w, mass_before;
};

__device__ __forceinline__ Fine fine_of(int bin, uint32_t sums, int C, uint32_t cnt0, unsigned long long mass0,
                                        const Softmax& sm) {
    const int lane = threadIdx.x & 31;
    Fine f;
    f.key = static_cast<uint32_t>(bin * 32 + 31 - lane);
    f.count = ld_dsmem_u32(map_peer(sums + ((bin / C) * 32 + 31 - lane) * 4, bin % C));
    f.w = f.count != 0 ? sm.fixed(f.key) : 0;
    uint32_t c = f.count;
    unsigned long long m = f.w * f.count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t cc = __shfl_up_sync(0xffffffffu, c, o);
        const unsigned long long mm = __shfl_up_sync(0xffffffffu, m, o);
        if (lane >= o) {
            c += cc;
            m += mm;
        }
    }
    f.count_before = cnt0 + c - f.count;
    f.mass_before = mass0 + m - f.w * f.count;
    return f;
}

// ---------------------------------------------------------------------------------------- window
constexpr int kWindowThreads = 256;
constexpr int kWindow = 4096;      // values counted below (and with) the largest, 16 a thread
constexpr int kUndone = -2;        // token of a row that is left to the counting kernel
constexpr int kVectors = 4;        // vectors of 8 logits a thread loads at a time
constexpr float kSmallWeight = 7.62939453125e-6f;  // 2^-17: 2^40 times less is below 2^23, exact in an fp32
constexpr float kTopWeight = 0.0009765625f;        // 2^-10: positions of likelier tokens are noted in passing

struct WindowShared {
    uint32_t kmax, threshold;
    uint32_t cut_at;           // a thread's answer
    unsigned long long cut_mass;
    unsigned long long tail;   // rank 0: mass below the window
    uint32_t warp_key[16];
    uint32_t warp_count[16];
    unsigned long long warp_mass[16];
    unsigned long long warp_tail[16];
    uint32_t pick_key, pick_index, pick_rank;
};
// counts, positions and weights of the window's values, largest first
constexpr size_t kWindowSmem = 1024 + kWindow * 12;

__device__ __forceinline__ void add_dsmem_u32_if(bool yes, uint32_t addr, uint32_t v) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p red.relaxed.cluster.shared::cluster.add.u32 [%1], %2;\n\t}" ::"r"(
            static_cast<uint32_t>(yes)),
        "r"(addr), "r"(v)
        : "memory");
}
__device__ __forceinline__ void st_dsmem_u32_if(bool yes, uint32_t addr, uint32_t v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p st.shared::cluster.u32 [%1], %2;\n\t}" ::"r"(
                     static_cast<uint32_t>(yes)),
                 "r"(addr), "r"(v)
                 : "memory");
}
__device__ __forceinline__ void add_dsmem_u64(uint32_t addr, unsigned long long v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// Where the `index`-th (from 0, in index order) occurrence of `key` is in elements begin .. end-1 of a
// row: written to *token by the thread that finds it. All threads of the CTA; scratch: 1024 words.
template <int kThreads>
__device__ __forceinline__ void find_occurrence(const uint16_t* src, int begin, int end, uint32_t key, uint32_t index,
                                                uint32_t* scratch, int32_t* token) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // vectors of 8 from the 16-byte boundary at or before the slice; elements outside it do not match
    const int base = begin - static_cast<int>((reinterpret_cast<uintptr_t>(src + begin) & 15u) / 2);
    const int total = (end - base + 7) / 8;
    const int per_warp = (total + kThreads / 32 - 1) / (kThreads / 32);
    const int v0 = min(total, warp * per_warp), v1 = min(total, v0 + per_warp);
    auto fetch = [&](int v) -> uint4 {
        const int i = base + 8 * v;
        if (v < v1 && i >= begin && i + 8 <= end) return *reinterpret_cast<const uint4*>(src + i);
        uint32_t w[4] = {0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u};
        if (v < v1)
            for (int j = 0; j < 8; ++j)
                if (i + j >= begin && i + j < end)
                    w[j / 2] = (j & 1) ? (w[j / 2] & 0xFFFFu) | (static_cast<uint32_t>(src[i + j]) << 16)
                                       : (w[j / 2] & 0xFFFF0000u) | src[i + j];
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    // compared as numbers: +0 and -0 are one value, NaN is none
    const __half2 value = __float2half2_rn(value_of(key));
    auto equal = [&](uint32_t w) { return __heq2(*reinterpret_cast<const __half2*>(&w), value); };  // 1 or 0
    auto bits_of = [&](const uint4& x) -> uint32_t {  // a bit for each of the vector's elements with the value
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __half2 e = equal(w[j]);
            bits |= (__low2float(e) != 0.f ? 1u << (2 * j) : 0u) | (__high2float(e) != 0.f ? 2u << (2 * j) : 0u);
        }
        return bits;
    };
    // a warp's share in rounds of 256 vectors (V <= 1,000,000: at most 62): how many in each
    constexpr int kRound = 8;
    __syncthreads();
    uint32_t count = 0;
    for (int v = v0, round = 0; v < v1; v += 32 * kRound, ++round) {
        uint4 x[kRound];
#pragma unroll
        for (int k = 0; k < kRound; ++k) x[k] = fetch(v + 32 * k + lane);
        __half2 n = __float2half2_rn(0.f);  // (32 of each half at most)
#pragma unroll
        for (int k = 0; k < kRound; ++k)
            n = __hadd2(n, __hadd2(__hadd2(equal(x[k].x), equal(x[k].y)), __hadd2(equal(x[k].z), equal(x[k].w))));
        if (lane == 0) scratch[warp * (32768 / kThreads) + round] = count;
        count += __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(__low2float(n) + __high2float(n)));
    }
    __syncwarp();
    __shared__ uint32_t totals[kThreads / 32];
    if (lane == 0) totals[warp] = count;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < warp; ++i) before += totals[i];
    if (index < before || index >= before + count) return;
    int round = 0;
    while (v0 + 32 * kRound * (round + 1) < v1 && before + scratch[warp * (32768 / kThreads) + round + 1] <= index) ++round;
    before += scratch[warp * (32768 / kThreads) + round];
    uint4 x[kRound];
#pragma unroll
    for (int k = 0; k < kRound; ++k) x[k] = fetch(v0 + 32 * kRound * round + 32 * k + lane);
#pragma unroll
    for (int k = 0; k < kRound; ++k) {
        const uint32_t bits = bits_of(x[k]), n = __popc(bits);
        uint32_t upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        if (index >= before + upto - n && index < before + upto)  // in this lane's vector
            *token = base + 8 * (v0 + 32 * kRound * round + 32 * k + lane) +
                     static_cast<int>(__fns(bits, 0, static_cast<int>(index - (before + upto - n)) + 1));
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
}

__global__ void __launch_bounds__(kWindowThreads, 4)
    sample_window_kernel(const uint16_t* __restrict__ logits, int64_t stride, int V, int slice,
                         const float* __restrict__ temperature, const int32_t* __restrict__ top_k,
                         const float* __restrict__ top_p, const float* __restrict__ min_p, const float* __restrict__ u,
                         int32_t* __restrict__ tokens, float* __restrict__ probs, int C, unsigned* status) {
    constexpr int kThreads = kWindowThreads;
    extern __shared__ __align__(16) uint8_t smem[];
    WindowShared& sh = *reinterpret_cast<WindowShared*>(smem);
    uint32_t* hist = reinterpret_cast<uint32_t*>(smem + 1024);
    uint32_t* where = hist + kWindow;
    float* weights = reinterpret_cast<float*>(where + kWindow);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_ctarank();
    const int64_t row = blockIdx.x / C;
    if (tid == 0) sh.tail = 0;
    weights[tid] = 0.f;  // (group maxima)
    griddep_launch_dependents();
    for (int i = tid; i < kWindow / 4; i += kThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    griddep_wait();
    const float t = temperature != nullptr ? temperature[row] : 1.f;
    const bool greedy = t <= 0.f;
    const int32_t kk = greedy ? 1 : (top_k != nullptr ? top_k[row] : 0);
    const float pp = top_p != nullptr ? top_p[row] : 1.f, mp = min_p != nullptr ? min_p[row] : 0.f, uu = u[row];

    // ---- first pass: the largest logit
    const int begin = min(V, static_cast<int>(rank) * slice), end = min(V, begin + slice);
    const uint16_t* src = logits + row * stride;
    const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(src + begin) & 15u) / 2);
    const int first = min(end, begin + (skew ? 8 - skew : 0));  // first element on a 16-byte boundary
    const int vectors = (end - first) / 8, last = first + 8 * vectors;
    const uint16_t* aligned = src + first;
    // the elements before and after the vectors: one each for the first few threads, masked elsewhere
    const uint32_t loose = tid < first - begin ? src[begin + tid]
                           : tid >= 8 && tid < 8 + end - last ? src[last + tid - 8] : 0xFC00u;
    const bool one_batch = vectors <= kVectors * kThreads;
    uint4 v[kVectors];
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < kVectors; ++k)
            v[k] = i0 + k * kThreads < vectors && in_bounds(first + 8 * (i0 + k * kThreads) + 8 <= V, status)
                       ? *reinterpret_cast<const uint4*>(aligned + 8 * static_cast<int64_t>(i0 + k * kThreads))
                       : make_uint4(0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u);
    };
    auto h2 = [](uint32_t w) { return *reinterpret_cast<const __half2*>(&w); };
    __half2 big = h2(0xFC00FC00u);
    for (int i0 = tid; i0 - tid < vectors; i0 += kVectors * kThreads) {
        load(i0);
#pragma unroll
        for (int k = 0; k < kVectors; ++k)
            big = __hmax2(big, __hmax2(__hmax2(h2(v[k].x), h2(v[k].y)), __hmax2(h2(v[k].z), h2(v[k].w))));
    }
    const uint32_t big_bits = *reinterpret_cast<const uint32_t*>(&big);
    uint32_t kmax = max(max(key_of(big_bits & 0xFFFFu), key_of(big_bits >> 16)), key_of(loose));
    // Small k: the cluster's elements in at least k groups (warps, or threads where there are more groups
    // than warps); the smallest of the groups' maxima has k tokens at or above it, and nothing below it matters.
    const int groups = (kk + C - 1) / C;
    const bool few = kk > 0 && kk <= kThreads && groups <= kThreads / 2;
    const bool by_warp = groups <= kThreads / 32;
    if (few && !by_warp) atomicMax(reinterpret_cast<uint32_t*>(weights) + tid % groups, kmax);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if (lane == 0) sh.warp_key[warp] = kmax;
    __syncthreads();
    uint32_t threshold = 0xFFFFu;
    if (few && by_warp) {
        uint32_t k = lane < groups ? 0 : 0xFFFFu;
        for (int i = lane; i < kThreads / 32 && lane < groups; i += groups) k = max(k, sh.warp_key[i]);
        threshold = k;
    } else if (few) {
        for (int i = lane; i < groups; i += 32) threshold = min(threshold, reinterpret_cast<const uint32_t*>(weights)[i]);
    }
    threshold = few ? __reduce_min_sync(0xffffffffu, threshold) : 0;
    for (int i = 0; i < kThreads / 32; ++i) kmax = max(kmax, sh.warp_key[i]);
    if (C > 1) {
        if (tid == 0) {
            sh.kmax = kmax;
            sh.threshold = threshold;
        }
        __syncwarp();
        cluster_sync_all();
        for (int r = 0; r < C; ++r) {
            kmax = max(kmax, ld_dsmem_u32(map_peer(smem_u32(&sh.kmax), r)));
            threshold = min(threshold, ld_dsmem_u32(map_peer(smem_u32(&sh.threshold), r)));
        }
    }
    if (kmax <= kMaskedKey) {  // nothing to choose from (no CTA of the row gets further)
        if (C > 1) cluster_sync_all();
        if (rank == 0 && tid == 0) {
            tokens[row] = -1;
            if (probs != nullptr) probs[row] = 0.f;
        }
        return;
    }
    Softmax sm;
    sm.kmax = kmax;
    sm.vmax = value_of(kmax);
    sm.temp = greedy ? 1.f : fminf(t, FLT_MAX);  // (infinite: every weight is 1, as with the largest)

    // ---- the window: unmasked values of the kWindow up to kmax, no lower than the cuts look
    uint32_t bottom = kmax >= kWindow + kMaskedKey ? kmax - kWindow + 1 : kMaskedKey + 1;
    const bool by_min = !(pp < 1.f) && mp > 0.f;
    if (few) bottom = max(bottom, threshold);
    const uint32_t low = mp > 0.f ? smallest_key(sm, fminf(mp, 1.f)) : 0;
    const bool enough = (few && bottom == max(threshold, kMaskedKey + 1)) || (by_min && low >= bottom);
    if (by_min) bottom = max(bottom, low);
    const uint32_t size = kmax - bottom + 1;
    // complete: nothing below the window can be kept, or count in the mass of those that are
    const bool complete = enough || bottom == kMaskedKey + 1 || sm.fixed(bottom - 1) == 0;
    const bool with_tail = !complete && !(kk > 0 && kk <= kWindow / 2);
    // Few elements are counted, and only rank 0 needs the counts: they go there directly.
    const bool sparse = C > 1 && enough;
    const bool tail_small = with_tail && sm.weight(bottom - 1) < kSmallWeight;

    // ---- second pass: count the window's values, note where likely ones are, add up the rest
    const float least = value_of(bottom), likely = fmaxf(least, value_of(smallest_key(sm, kTopWeight)));
    const float r_temp = 1.f / sm.temp;
    const bool unit = sm.temp == 1.f;
    const uint32_t hist_s = smem_u32(hist), hist_0 = C > 1 ? map_peer(hist_s, 0) : hist_s;
    const uint32_t where_0 = sparse ? map_peer(smem_u32(where), 0) : smem_u32(where);
    unsigned long long tail = 0;
    const __half2 zero = h2(0u);
    auto clean = [&](uint32_t w) {  // -0 becomes 0, every NaN the positive one (whose key is above all)
        const __half2 x = __hadd2(h2(w), zero);
        return *reinterpret_cast<const uint32_t*>(&x);
    };
    auto below = [&](uint32_t bits) {  // places below the largest; wraps for NaN
        const uint32_t neg = static_cast<uint32_t>(static_cast<int>(bits << 16) >> 31);
        return kmax - ((bits ^ (neg | 0x8000u)) & 0xFFFFu);
    };
    // Without a branch: what is not counted goes to a word of the thread's own (256 rows 120 us with a predicate)
    const uint32_t aside = smem_u32(weights) + (kThreads + tid) * 4;
    auto count_one = [&](uint32_t d) {
        asm volatile("red.shared::cta.add.u32 [%0], 1;" ::"r"(d < size ? hist_s + d * 4 : aside) : "memory");
    };
    auto half_of = [](uint32_t bits) { return __half2float(__ushort_as_half(static_cast<unsigned short>(bits))); };
    auto exponent = [&](float x) {  // weight of a logit below the window
        float z = __fsub_rn(x, sm.vmax);
        if (!unit) {  // z / temp: quotient by the reciprocal and one correction (Markstein 1990)
            const float q = __fmul_rn(z, r_temp);
            z = __fmaf_rn(__fmaf_rn(-q, sm.temp, z), r_temp, q);
        }
        return expf(fmaxf(z, -200.f));  // (NaN and -inf: weight 0)
    };
    // 2^40 times a weight below 2^-17: rounded by adding 2^23
    auto small_fixed_of = [&](float w, float unit_of) { return __float_as_uint(__fmaf_rn(w, unit_of, 8388608.f)) - 0x4B000000u; };
    // 2^40 times any weight: whole 2^20s and the rest, each exact or rounded once
    auto add_fixed = [&](float w, uint32_t& high, uint32_t& low) {
        const float a = __fmul_rn(w, 1048576.f), h = __fadd_rz(a, 8388608.f);
        high += __float_as_uint(h) - 0x4B000000u;
        low += small_fixed_of(__fsub_rn(a, __fsub_rn(h, 8388608.f)), 1048576.f);
    };
    // Notes the positions of a vector's likely elements, and counts a sparse row's. Called by whole warps and
    // without branches: a lane whose vector has none goes along. (With a branch a lane for each element the
    // lanes of a warp took turns: a row with 15,660 likely tokens cost 870 us instead of 100.)
    auto note = [&](const uint4& x, int index) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t bits = (j & 1) ? w[j / 2] >> 16 : w[j / 2] & 0xFFFFu;
            const uint32_t d = below(clean(bits) & 0xFFFFu);
            if (sparse) add_dsmem_u32_if(d < size, hist_0 + d * 4, 1u);
            st_dsmem_u32_if(half_of(bits) >= likely, where_0 + d * 4, index + j);
        }
    };
    for (int i0 = tid; i0 - tid < vectors; i0 += kVectors * kThreads) {
        if (!one_batch) load(i0);
        uint32_t part = 0, high = 0;  // 32 weights below 2^23; or their whole 2^20s and the rest
#pragma unroll
        for (int k = 0; k < kVectors; ++k) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            const __half2 m = __hmax2(__hmax2(h2(w[0]), h2(w[1])), __hmax2(h2(w[2]), h2(w[3])));
            const float top = fmaxf(__low2float(m), __high2float(m));
            if (__any_sync(0xffffffffu, top >= (sparse ? least : likely))) note(v[k], first + 8 * (i0 + k * kThreads));
            if (tail_small) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t b = clean(w[j]), d0 = below(b & 0xFFFFu), d1 = below(b >> 16);
                    count_one(d0);
                    count_one(d1);
                    const float x0 = d0 < size ? -INFINITY : half_of(b & 0xFFFFu), x1 = d1 < size ? -INFINITY : half_of(b >> 16);
                    part += small_fixed_of(exponent(x0), 1099511627776.f) + small_fixed_of(exponent(x1), 1099511627776.f);
                }
            } else if (with_tail) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t b = clean(w[j]), d0 = below(b & 0xFFFFu), d1 = below(b >> 16);
                    count_one(d0);
                    count_one(d1);
                    const float x0 = d0 < size ? -INFINITY : half_of(b & 0xFFFFu), x1 = d1 < size ? -INFINITY : half_of(b >> 16);
                    add_fixed(exponent(x0), high, part);
                    add_fixed(exponent(x1), high, part);
                }
            } else if (!sparse && top >= least) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t b = clean(w[j]);
                    count_one(below(b & 0xFFFFu));
                    count_one(below(b >> 16));
                }
            }
        }
        tail += part + (static_cast<unsigned long long>(high) << 20);
    }
    {
        const uint32_t bits = clean(loose) & 0xFFFFu, d = below(bits);
        if (sparse) {
            add_dsmem_u32_if(d < size, hist_0 + d * 4, 1u);
        } else {
            count_one(d);
        }
        if (with_tail && d >= size) tail += __float2ull_rn(exponent(half_of(bits)) * 1099511627776.f);
        st_dsmem_u32_if(half_of(bits) >= likely, where_0 + d * 4, tid < 8 ? begin + tid : last + tid - 8);
    }
    if (with_tail) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) tail += __shfl_xor_sync(0xffffffffu, tail, o);
        if (lane == 0) sh.warp_tail[warp] = tail;
    }
    __syncthreads();
    if (tid == 0 && with_tail) {
        tail = 0;
        for (int i = 0; i < kThreads / 32; ++i) tail += sh.warp_tail[i];
        add_dsmem_u64(map_peer(smem_u32(&sh.tail), 0), tail);
    }
    if (sparse) {
        __syncwarp();
        cluster_sync_all();
        if (rank != 0) return;  // rank 0 needs nothing more of the others
    } else if (C > 1) {  // rank r adds up its share of the counts, into rank 0's weights array (not in use yet)
        __syncwarp();
        cluster_sync_all();
        const int share = kWindow / C;
        for (int i = static_cast<int>(rank) * share + 4 * tid; i < (static_cast<int>(rank) + 1) * share; i += 4 * kThreads) {
            uint4 n = make_uint4(0, 0, 0, 0);
            for (int r = 0; r < C; ++r) {
                const uint4 x = ld_dsmem_u4(map_peer(hist_s + i * 4, r));
                n.x += x.x;
                n.y += x.y;
                n.z += x.z;
                n.w += x.w;
            }
            st_dsmem_u4(map_peer(smem_u32(weights + i), 0), n);
        }
        __syncwarp();
        cluster_sync_all();
    } else {
        __syncthreads();
    }

    if (rank == 0) {
        // ---- weights and running sums: thread t has `per` values from per * t below the largest. (Of rank
        // 0's own counts in a cluster nothing is needed any more: the weights take their place.)
        const bool added = C > 1 && !sparse;
        const uint32_t* counts = added ? reinterpret_cast<const uint32_t*>(weights) : hist;
        float* w_of = added ? reinterpret_cast<float*>(hist) : weights;
        const uint32_t per = (size + kThreads - 1) / kThreads;
        const uint32_t d0 = min(size, tid * per), d1 = min(size, d0 + per);
        uint32_t count = 0;
        unsigned long long mass = 0, by_weight = 0;  // by_weight: of values with weight >= min_p
        for (uint32_t i = 0, at = lane % per; i < per; ++i, at = at + 1 == per ? 0 : at + 1) {
            const uint32_t d = d0 + at;  // (each lane begins elsewhere: no bank conflicts)
            const uint32_t n = d < d1 ? counts[d] : 0;
            if (n == 0) continue;
            const float w = sm.weight(kmax - d);
            const unsigned long long m = n * __float2ull_rn(w * 1099511627776.f);
            w_of[d] = w;
            count += n;
            mass += m;
            if (w >= mp) by_weight += m;
        }
        auto fixed_at = [&](uint32_t d) { return __float2ull_rn(w_of[d] * 1099511627776.f); };
        uint32_t cs = count;
        unsigned long long ms = mass;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t cc = __shfl_up_sync(0xffffffffu, cs, o);
            const unsigned long long mm = __shfl_up_sync(0xffffffffu, ms, o);
            if (lane >= o) {
                cs += cc;
                ms += mm;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) by_weight += __shfl_xor_sync(0xffffffffu, by_weight, o);
        if (lane == 31) {
            sh.warp_count[warp] = cs;
            sh.warp_mass[warp] = ms;
            sh.warp_tail[warp] = by_weight;
        }
        __syncthreads();
        uint32_t cb = cs - count, counted = 0;
        unsigned long long mb = ms - mass, window_mass = 0;
        by_weight = 0;
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) {
                cb += sh.warp_count[i];
                mb += sh.warp_mass[i];
            }
            counted += sh.warp_count[i];
            window_mass += sh.warp_mass[i];
            by_weight += sh.warp_tail[i];
        }
        constexpr unsigned long long kOne = 1ull << 40;  // the first token
        bool undone = false;
        unsigned long long all = window_mass + sh.tail;
        if (kk > 0 && static_cast<uint32_t>(kk) < counted) {
            const uint32_t k = kk;
            if (cb < k && k <= cb + count) {  // the k-th token is one of this thread's values
                uint32_t c = cb;
                unsigned long long m = mb;
                for (uint32_t d = d0; d < d1 && c < k; ++d) {
                    const uint32_t n = min(counts[d], k - c);
                    if (n != 0) m += n * fixed_at(d);
                    c += n;
                }
                sh.cut_mass = m;
            }
            __syncthreads();
            all = sh.cut_mass;
        } else if (kk > 0 && static_cast<uint32_t>(kk) != counted && !complete) {
            undone = true;  // the k-th token is below the window
        } else if (kk > 0 && static_cast<uint32_t>(kk) == counted) {
            all = window_mass;
        }
        unsigned long long kept = all;
        if (pp < 1.f) {
            const unsigned long long limit = scaled(all, static_cast<unsigned long long>(fmaxf(pp, 0.f) * 16777216.f));
            if (limit > window_mass) {
                undone = true;
            } else if (limit == 0) {
                kept = kOne;
            } else {
                __syncthreads();
                if (mb < limit && limit <= mb + mass) {  // the running mass reaches the limit in this thread's values
                    unsigned long long m = mb;
                    for (uint32_t d = d0; d < d1 && m < limit; ++d) {
                        const unsigned long long n = counts[d], w = n != 0 ? fixed_at(d) : 0;
                        if (n * w < limit - m) m += n * w;
                        else m += (limit - m + w - 1) / w * w;
                    }
                    sh.cut_mass = m;
                }
                __syncthreads();
                kept = min(kept, sh.cut_mass);
            }
        }
        if (mp > 0.f) {
            if (low < bottom && !complete && kept > window_mass) undone = true;  // the cut is below the window
            kept = min(kept, max(by_weight, kOne));
        }
        const unsigned long long x =
            scaled(kept, static_cast<unsigned long long>(fminf(fmaxf(uu * 16777216.f, 0.f), 16777215.f)));
        if (x >= window_mass) undone = true;  // drawn from below the window
        if (tid == 0) sh.pick_key = 0;
        __syncthreads();
        if (undone) {
            if (tid == 0) tokens[row] = kUndone;
        } else if (mb <= x && x < mb + mass) {
            unsigned long long m = mb;
            for (uint32_t d = d0; d < d1; ++d) {
                const uint32_t n = counts[d];
                if (n == 0) continue;
                const unsigned long long w = fixed_at(d);
                if (x < m + n * w) {
                    if (probs != nullptr) probs[row] = static_cast<float>(static_cast<double>(w) / static_cast<double>(kept));
                    sh.pick_index = static_cast<uint32_t>((x - m) / w);
                    sh.pick_key = kmax - d;
                    sh.cut_at = n;
                    break;
                }
                m += n * w;
            }
        }
        __syncthreads();
        if (added && warp == 0) {  // which CTA's slice has that occurrence
            const uint32_t key = sh.pick_key, d = kmax - key;
            uint32_t here = key != 0 && lane > 0 && lane < C ? ld_dsmem_u32(map_peer(hist_s + d * 4, lane)) : 0;
            const uint32_t others = __reduce_add_sync(0xffffffffu, here);
            if (lane == 0 && key != 0) here = sh.cut_at - others;
            uint32_t upto = here;
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            const uint32_t index = sh.pick_index;
            __syncwarp();
            if (lane < C) {
                const bool owner = key != 0 && index >= upto - here && index < upto;
                st_dsmem_u32(map_peer(smem_u32(&sh.pick_rank), lane), owner ? 1u : 0u);
                if (owner) {
                    const uint32_t local = index - (upto - here);
                    st_dsmem_u32(map_peer(smem_u32(&sh.cut_at), lane), here);
                    if (lane != 0) st_dsmem_u32(map_peer(smem_u32(&sh.pick_key), lane), key);
                    st_dsmem_u32(map_peer(smem_u32(&sh.pick_index), lane), local);
                }
            }
        } else if (!added && tid == 0) {
            sh.pick_rank = sh.pick_key != 0;
        }
    }
    if (C > 1 && !sparse) {
        __syncwarp();
        cluster_sync_all();
    } else {
        __syncthreads();
    }
    if (sh.pick_rank == 0) return;
    const uint32_t key = sh.pick_key;
    if (sh.cut_at == 1 && value_of(key) >= likely) {  // noted in passing
        if (tid == 0) tokens[row] = static_cast<int32_t>(where[kmax - key]);
        return;
    }
    // (a sparse row's is looked for by rank 0 in the whole row: equal logits among its few likely tokens)
    find_occurrence<kThreads>(src, sparse ? 0 : begin, sparse ? V : end, key, sh.pick_index, reinterpret_cast<uint32_t*>(weights), tokens + row);
}

// -------------------------------------------------------------------------------------- counting
struct Shared {  // at the start of dynamic shared memory, before the arrays
    uint32_t kmax;
    uint32_t pick_key, pick_index;
    int pick_owner;
    uint32_t warp_count[kThreads / 32];
    unsigned long long warp_mass[kThreads / 32];
    uint32_t warp_key[kThreads / 32];
};

__global__ void __launch_bounds__(kThreads, 1)
    sample_kernel(const uint16_t* __restrict__ logits, int64_t stride, int V, int slice,
                  const float* __restrict__ temperature, const int32_t* __restrict__ top_k,
                  const float* __restrict__ top_p, const float* __restrict__ min_p, const float* __restrict__ u,
                  int32_t* __restrict__ tokens, float* __restrict__ probs, int C, unsigned* status) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    uint32_t* hist = reinterpret_cast<uint32_t*>(smem + 1024);  // two 16-bit counters a word
    unsigned long long* all_mass = reinterpret_cast<unsigned long long*>(smem + 1024 + kHistBytes);
    uint32_t* all_count = reinterpret_cast<uint32_t*>(all_mass + kBins);
    uint32_t* sums = all_count + kBins;  // the cluster's counts of this CTA's bins: bin rank + C i at 32 i
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_ctarank();
    const int64_t row = blockIdx.x / C;

    griddep_launch_dependents();
    griddep_wait();
    if (tokens[row] != kUndone) return;  // (the whole cluster)
    for (int i = tid; i < static_cast<int>(kHistBytes / 16); i += kThreads)
        reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();

    // ---- one pass over this CTA's slice: count the values, find the largest
    const int begin = min(V, static_cast<int>(rank) * slice), end = min(V, begin + slice);
    const uint16_t* src = logits + row * stride;
    uint32_t kmax = 0;
    auto take = [&](uint32_t bits) {
        const uint32_t key = key_of(bits);
        if (key > kMaskedKey) {
            kmax = max(kmax, key);
            atomicAdd(&hist[key >> 1], (key & 1u) ? 65536u : 1u);
        }
    };
    const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(src + begin) & 15u) / 2);
    const int first = min(end, begin + (skew ? 8 - skew : 0));  // first element on a 16-byte boundary
    const int vectors = (end - first) / 8;
    if (tid < first - begin) take(src[begin + tid]);
    // loads of 8 vectors a thread before their first count: one trip to memory for 64 elements
    for (int i0 = tid; i0 < vectors; i0 += 8 * kThreads) {
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i0 + k * kThreads < vectors && in_bounds(first + 8 * (i0 + k * kThreads) + 8 <= V, status))
                v[k] = *reinterpret_cast<const uint4*>(src + first + 8 * static_cast<int64_t>(i0 + k * kThreads));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (i0 + k * kThreads >= vectors) break;
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                take(w[j] & 0xFFFFu);
                take(w[j] >> 16);
            }
        }
    }
    if (tid < end - first - 8 * vectors) take(src[first + 8 * vectors + tid]);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if (lane == 0) sh.warp_key[warp] = kmax;
    __syncthreads();
    if (tid == 0) {
        for (int i = 1; i < kThreads / 32; ++i) kmax = max(kmax, sh.warp_key[i]);
        sh.kmax = kmax;
        sh.pick_owner = -1;  // until rank 0 names the CTA that holds the chosen token
    }
    cluster_sync_all();
    kmax = 0;
    for (int r = 0; r < C; ++r) kmax = max(kmax, ld_dsmem_u32(map_peer(smem_u32(&sh.kmax), r)));

    Softmax sm;
    sm.kmax = kmax;
    sm.vmax = value_of(kmax);
    const float t = temperature != nullptr ? temperature[row] : 1.f;
    const bool greedy = t <= 0.f;
    sm.temp = greedy ? 1.f : fminf(t, FLT_MAX);  // (infinite: every weight is 1, as with the largest)

    // ---- the cluster's counts of this CTA's bins, a quarter of a bin a thread; their count and mass go to
    // rank 0. Values whose weight is 0 are left out (every cut among them leaves the masses as they are).
    const uint32_t hist_s = smem_u32(hist);
    for (int i = tid; i < kBins / C * 4; i += kThreads) {
        const int b = static_cast<int>(rank) + C * (i >> 2), k0 = b * 32 + (i & 3) * 8;
        uint32_t count = 0, n[8] = {};
        unsigned long long mass = 0;
        if (b * 32 <= static_cast<int>(kmax) && sm.fixed(min(kmax, static_cast<uint32_t>(b * 32 + 31))) != 0) {
            for (int r0 = 0; r0 < C; r0 += 4) {
                uint4 v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = ld_dsmem_u4(map_peer(hist_s + k0 * 2, r0 + r));
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t w[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        n[2 * j] += w[j] & 0xFFFFu;
                        n[2 * j + 1] += w[j] >> 16;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (n[j] == 0) continue;
                const unsigned long long w = sm.fixed(static_cast<uint32_t>(k0 + j));
                if (w == 0) n[j] = 0;
                count += n[j];
                mass += n[j] * w;
            }
        }
        uint4* to = reinterpret_cast<uint4*>(sums + i * 8);
        to[0] = make_uint4(n[0], n[1], n[2], n[3]);
        to[1] = make_uint4(n[4], n[5], n[6], n[7]);
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            count += __shfl_xor_sync(0xffffffffu, count, o);
            mass += __shfl_xor_sync(0xffffffffu, mass, o);
        }
        if ((i & 3) == 0) {
            st_dsmem_u32(map_peer(smem_u32(all_count + b), 0), count);
            st_dsmem_u64(map_peer(smem_u32(all_mass + b), 0), mass);
        }
    }
    cluster_sync_all();

    if (rank == 0) {
        // ---- what precedes each bin, bins in descending order: position i is bin kBins - 1 - i
        constexpr int kPer = kBins / kThreads;
        uint32_t c[kPer], ct = 0;
        unsigned long long m[kPer], mt = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = kBins - 1 - (tid * kPer + i);
            c[i] = all_count[b];
            m[i] = all_mass[b];
            ct += c[i];
            mt += m[i];
        }
        uint32_t cs = ct;
        unsigned long long ms = mt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t cc = __shfl_up_sync(0xffffffffu, cs, o);
            const unsigned long long mm = __shfl_up_sync(0xffffffffu, ms, o);
            if (lane >= o) {
                cs += cc;
                ms += mm;
            }
        }
        if (lane == 31) {
            sh.warp_count[warp] = cs;
            sh.warp_mass[warp] = ms;
        }
        __syncthreads();
        uint32_t cb = cs - ct, total_count = 0;
        unsigned long long mb = ms - mt, total_mass = 0;
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) {
                cb += sh.warp_count[i];
                mb += sh.warp_mass[i];
            }
            total_count += sh.warp_count[i];
            total_mass += sh.warp_mass[i];
        }
        uint32_t* bin_count = all_count;  // from here on what precedes a bin, in position order
        unsigned long long* bin_mass = all_mass;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            bin_count[tid * kPer + i] = cb;
            bin_mass[tid * kPer + i] = mb;
            cb += c[i];
            mb += m[i];
        }
        __syncthreads();
        if (warp == 0) {
            const uint32_t sums_s = smem_u32(sums);
            // last position whose preceding count / mass is <= x
            auto find = [&](auto* before, unsigned long long x) {
                int pos = (31 - __clz(__ballot_sync(0xffffffffu, before[64 * lane] <= x))) * 64;
                pos += (31 - __clz(__ballot_sync(0xffffffffu, before[pos + 2 * lane] <= x))) * 2;
                return before[pos + 1] <= x ? pos + 1 : pos;
            };
            auto at = [&](int pos) { return fine_of(kBins - 1 - pos, sums_s, C, bin_count[pos], bin_mass[pos], sm); };
            auto lane_of = [&](bool p) { return 31 - __clz(__ballot_sync(0xffffffffu, p)); };  // last lane
            if (total_count == 0) {
                if (lane == 0) {
                    tokens[row] = -1;
                    if (probs != nullptr) probs[row] = 0.f;
                }
            } else {
                // the kept prefix ends with `items` tokens of value `cut`
                uint32_t cut = 0, items = 0xFFFFFFFFu;
                unsigned long long mass = total_mass;
                const int32_t kk = greedy ? 1 : (top_k != nullptr ? top_k[row] : 0);
                if (kk > 0 && static_cast<uint32_t>(kk) < total_count) {
                    const Fine f = at(find(bin_count, static_cast<unsigned long long>(kk - 1)));
                    const int l = lane_of(f.count != 0 && f.count_before <= static_cast<uint32_t>(kk - 1));
                    cut = __shfl_sync(0xffffffffu, f.key, l);
                    items = kk - __shfl_sync(0xffffffffu, f.count_before, l);
                    mass = __shfl_sync(0xffffffffu, f.mass_before, l) + items * __shfl_sync(0xffffffffu, f.w, l);
                }
                const float p = top_p != nullptr ? top_p[row] : 1.f;
                if (p < 1.f) {
                    const unsigned long long limit =
                        scaled(mass, static_cast<unsigned long long>(fmaxf(p, 0.f) * 16777216.f));
                    if (limit == 0) {
                        cut = kmax;
                        items = 1;
                    } else {
                        const Fine f = at(find(bin_mass, limit - 1));
                        const int l = lane_of(f.w * f.count != 0 && f.mass_before <= limit - 1);
                        const unsigned long long w = __shfl_sync(0xffffffffu, f.w, l);
                        cut = __shfl_sync(0xffffffffu, f.key, l);
                        items = static_cast<uint32_t>((limit - 1 - __shfl_sync(0xffffffffu, f.mass_before, l)) / w) + 1;
                    }
                }
                const float mp = min_p != nullptr ? min_p[row] : 0.f;
                if (mp > 1.f) {
                    cut = kmax;
                    items = 1;
                } else if (mp > 0.f) {
                    const uint32_t base = smallest_key(sm, mp);  // the smallest value with weight >= min_p
                    if (base > cut) {
                        cut = base;
                        items = 0xFFFFFFFFu;
                    }
                }
                unsigned long long kept = total_mass;
                if (cut != 0) {
                    const int pos = kBins - 1 - static_cast<int>(cut >> 5);
                    const Fine f = at(pos);
                    const int l = 31 - static_cast<int>(cut & 31u);
                    const uint32_t n = min(items, __shfl_sync(0xffffffffu, f.count, l));
                    kept = __shfl_sync(0xffffffffu, f.mass_before, l) + n * __shfl_sync(0xffffffffu, f.w, l);
                }
                const float uu = u[row];
                const unsigned long long u24 =
                    static_cast<unsigned long long>(fminf(fmaxf(uu * 16777216.f, 0.f), 16777215.f));
                const unsigned long long x = scaled(kept, u24);
                const Fine f = at(find(bin_mass, x));
                const int l = lane_of(f.w * f.count != 0 && f.mass_before <= x);
                const uint32_t key = __shfl_sync(0xffffffffu, f.key, l);
                const unsigned long long w = __shfl_sync(0xffffffffu, f.w, l);
                uint32_t index = static_cast<uint32_t>((x - __shfl_sync(0xffffffffu, f.mass_before, l)) / w);
                // which CTA's slice holds occurrence `index` of the value
                uint32_t here = lane < C ? ld_dsmem_u16(map_peer(hist_s + key * 2, lane)) : 0, upto = here;
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) {
                    const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += v;
                }
                const int owner = __ffs(__ballot_sync(0xffffffffu, upto > index)) - 1;
                index -= __shfl_sync(0xffffffffu, upto - here, owner);
                if (lane < C) {
                    st_dsmem_u32(map_peer(smem_u32(&sh.pick_owner), lane), static_cast<uint32_t>(owner));
                    st_dsmem_u32(map_peer(smem_u32(&sh.pick_key), lane), key);
                    st_dsmem_u32(map_peer(smem_u32(&sh.pick_index), lane), index);
                }
                if (lane == 0 && probs != nullptr)
                    probs[row] = static_cast<float>(static_cast<double>(w) / static_cast<double>(kept));
            }
        }
    }
    __syncwarp();
    cluster_sync_all();
    if (sh.pick_owner != static_cast<int>(rank)) return;

    // ---- the owner finds occurrence pick_index of the value in its slice, in index order
    find_occurrence<kThreads>(src, begin, end, sh.pick_key, sh.pick_index, sums, tokens + row);
}

}  // namespace

namespace {

template <typename F>
cudaError_t launch_rows(F* f, const SampleParams& p, int C, int threads, size_t smem, cudaStream_t s, unsigned* status) {
    const int slice = ((p.V + C - 1) / C + 7) / 8 * 8;
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (C > 8) {
        e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(p.M) * C), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(C);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, f, p.logits, p.stride, p.V, slice, p.temperature, p.top_k, p.top_p, p.min_p, p.u,
                              p.tokens, p.probs, C, status);
}

}  // namespace

cudaError_t launch_sample(const SampleParams& p, int sm_count, cudaStream_t s, unsigned* status) {
    // Window: 256 threads, four CTAs an SM (with 512 and two, and 8192 values: 256 rows of 248,320 153 us
    // against then 139, 33 mixed rows of 32,003 26.7 against then 24.4). Few rows are spread over up to 16 CTAs
    // (1 row 12.2 us, with 8 14.0), more over up to 8 (16 rows 12.6, with 16 13.2), many over as many as make
    // two rounds (256 rows, of then 122 us with 4: 187 with 1, 141 with 2, 140 with 8).
    int C = p.M <= 8 ? 16 : 8;
    while (C > 1 && static_cast<int64_t>(p.M) * C > 7LL * sm_count) C /= 2;
    cudaError_t e = launch_rows(sample_window_kernel, p, C, kWindowThreads, kWindowSmem, s, status);
    if (e != cudaSuccess) return e;
    // Counting: one CTA an SM; enough a row that each counts fewer than 65,536 values.
    C = p.M <= 9 ? 16 : p.M <= 18 ? 8 : 4;
    while (C < 16 && (p.V + C - 1) / C > 65528) C *= 2;
    return launch_rows(sample_kernel, p, C, kThreads, kSmemBytes, s, status);
}

}  // namespace w4a16
