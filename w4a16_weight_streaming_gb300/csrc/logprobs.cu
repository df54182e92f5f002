// Log probabilities of rows of fp16 logits, in one pass over a row:
//
//   p_i = exp((l_i - l_max) / T) / S,  S = sum_i exp((l_i - l_max) / T)      (NaN and -inf: p = 0)
//   log p of given tokens, and their places in the order (logits descending, ties by lower index)
//   entropy  -sum p log p = log S - (1 / S) sum_i w_i d_i,  d_i = (l_i - l_max) / T, w_i = exp(d_i): two sums
//            of one sign, nothing cancels
//   the first n of the order
//
// A thread takes 32 neighbouring logits (a chunk, 64 bytes) at a time; it keeps the largest logit
// so far, S and sum w d relative to it, and rescales both when a larger one turns up. A masked logit is read
// as -65504, whose weight is 0 where the largest is not as low itself or T is below hundreds; elsewhere, and
// for infinite ones, a chunk goes the slow way, logit by logit.
//
// A place is a count: logits above the given one, and equal ones before it; "equal or above" is "above the
// next smaller fp16 number", so either is one packed comparison, its masks added up as whole numbers (3 instructions for
// 4 logits; 4 with fp16 counts: 1024 rows 5 us more), and a warp with no logit above skips it.
//
// The first n: each chunk leaves its maximum in shared memory. The first n of a row lie in the n chunks that
// come first in the order (maximum, then lower chunk): a chunk before another has an element before each of
// the other's. So a search among the maxima names n chunks, and only their n * 32 elements are read a
// second time.
//
// A row is a CTA or a cluster, whose parts rank 0 brings together in a fixed order. Many rows are a CTA of 128 threads
// each, seven an SM, so that 1024 rows run at once (256 threads, four an SM: a second, partial round, 110 us where 128
// took 103). While a warp works on its 32 chunks, its next ones are on their way into shared memory.
//
// Measured on one GB300, vocabulary 248,320, in a CUDA graph: 1024 rows, a token and the first alternative each, 89.5 us
// (509 MB, 5.7 TB/s, 0.84 of the measured copy) where some rows' tokens are unlikely, 84 where all are likely (no counting),
// 80 without token and alternatives: instructions beside the stream, 8 a logit with all of it (with the next chunk prefetched
// into L2 only 91.3; with (l - m) c in two instructions 97, with counts in fp16 and that 101). One row with 20
// alternatives 14.7 us, 16 rows with two tokens each 8.75, 33 rows of 32,003 with 5 alternatives 10.8: latency, of the
// launch, the token's logit, one chunk or two a thread, the search's six barriers and the cluster's two.
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {
namespace {

constexpr int kChunk = 32;       // elements, 64 bytes and on their boundary
constexpr int kCandidates = 1024;
constexpr int kMaxTop = 32;
constexpr uint32_t kMasked2 = 0xFC00FC00u;  // (-inf, -inf)

struct LogprobArgs {
    const uint16_t* logits;
    int64_t stride;
    int V;
    const int32_t* tokens;  // [M][given]
    int given, top;
    const float* temperature;
    float* logprob;
    int32_t* rank;
    float* entropy;
    int32_t* top_tokens;
    float* top_logprob;
};

struct Sums {
    float m, s, d;  // largest logit, sum of weights, sum of weight * exponent (in powers of 2)
};

template <int NG, int kThreads>
struct __align__(16) Shared {
    static constexpr int kWarps = kThreads / 32;
    unsigned long long best[kMaxTop];          // this CTA's first tokens
    union {
        unsigned long long cand[kCandidates];  // (value key, ~index)
        uint4 next[kWarps][128];               // before: each warp's next 32 chunks
    };
    uint32_t keys[kCandidates];                // (value key of a chunk's maximum, ~chunk)
    uint32_t first[kThreads];                  // the first of each thread's maxima
    uint32_t least;
    uint32_t chunk[kMaxTop];
    uint32_t last;                             // value key of the n-th chunk
    int count, found;
    Sums part[kWarps];
    uint32_t above[kWarps][NG == 0 ? 1 : NG];
    Sums whole;                                // of this CTA
    uint32_t above_whole[NG == 0 ? 1 : NG];
    uint32_t given[NG == 0 ? 1 : NG];  // bits of a given token's logit, with how many of its chunk before it equal it << 16
};

// Order of the numbers as 16 bits, above 0; 0 for a masked one. -0 and 0 are one value.
__device__ __forceinline__ uint32_t key_of(uint32_t bits) {
    if ((bits & 0x7FFFu) > 0x7C00u || bits == 0xFC00u) return 0u;
    if (bits == 0x8000u) bits = 0;
    return (bits & 0x8000u) ? (~bits & 0xFFFFu) : (bits | 0x8000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    const uint32_t bits = (key & 0x8000u) ? (key & 0x7FFFu) : (~key & 0xFFFFu);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}
__device__ __forceinline__ uint32_t below(uint32_t bits) {  // the next smaller fp16 number (of a finite one or +inf)
    return (bits & 0x7FFFu) == 0 ? 0x8001u : (bits & 0x8000u) ? bits + 1 : bits - 1;
}

__device__ __forceinline__ void ldg_stream(uint32_t* v, const void* p) {  // 32 bytes, aligned to them
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
}
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Exponents are those of 2, relative to the largest logit m: l c - k with k = m c rounded, one fused multiply-add a logit; what
// the rounding of k makes of all weights is taken out at the end. Where k may be too large for that (`far`: T below 0.09),
// (l - m) c.
struct Scale {
    float c;
    bool far;
    __device__ __forceinline__ float from(float l, float m) const { return far ? (l - m) * c : fmaf(l, c, -__fmul_rn(m, c)); }
    __device__ __forceinline__ float between(float m0, float m1) const {
        return far ? (m0 - m1) * c : __fsub_rn(__fmul_rn(m0, c), __fmul_rn(m1, c));
    }
};

// `a` seen from the larger maximum m.
__device__ __forceinline__ void rescale(Sums& a, float m, const Scale& c) {
    if (a.s == 0.f) {
        a.d = 0.f;
    } else if (m == INFINITY) {
        if (a.m != m) a.s = a.d = 0.f;
    } else {
        const float x = c.between(a.m, m), e = ex2(x);
        a.d = e == 0.f ? 0.f : e * fmaf(x, a.s, a.d);
        a.s *= e;
    }
    a.m = m;
}
__device__ __forceinline__ Sums joined(Sums a, Sums b, const Scale& c) {
    const float m = fmaxf(a.m, b.m);
    rescale(a, m, c);
    rescale(b, m, c);
    return {m, a.s + b.s, a.d + b.d};
}

__device__ __forceinline__ Sums shuffled(const Sums& a, int o) {
    return {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o), __shfl_xor_sync(0xffffffffu, a.d, o)};
}

// How many of n sorted keys (descending) are above k.
__device__ __forceinline__ int above_in(const unsigned long long* sorted, int n, unsigned long long k) {
    int at = 0;
#pragma unroll
    for (int step = 32; step > 0; step >>= 1)
        if (at + step <= n && sorted[at + step - 1] > k) at += step;
    return at;
}

template <int NG, bool TOP, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) logprobs_kernel(const LogprobArgs a, int C, int64_t total, unsigned* status) {
    extern __shared__ __align__(16) uint16_t chunk_max[];  // fp16 maxima of this CTA's chunks
    constexpr int kWarps = kThreads / 32;
    __shared__ Shared<NG, kThreads> sh;
    constexpr int kG = NG == 0 ? 1 : NG;
    griddep_launch_dependents();
    const int rank = static_cast<int>(blockIdx.x) % C, m = static_cast<int>(blockIdx.x) / C;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint16_t* row = a.logits + static_cast<int64_t>(m) * a.stride;
    // Chunk i holds elements 32 i - off and on, 64-byte aligned; the first and last may lie outside the row in part.
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) >> 1) & 31u);
    const unsigned char* chunk0 = reinterpret_cast<const unsigned char*>(row - off);
    const int chunks_all = (off + a.V + 31) / 32, per = (chunks_all + C - 1) / C;
    const int c0 = min(chunks_all, rank * per), c1 = min(chunks_all, c0 + per);
    const int inner0 = off == 0 ? 0 : 1, inner1 = (off + a.V) / 32;  // whole chunks
    uint32_t x[16];
    auto load = [&](int i) {
        if (i >= inner0 && i < min(c1, inner1) && in_bounds(m * a.stride + 32LL * i - off + 32 <= total, status)) {
            ldg_stream(x, chunk0 + static_cast<int64_t>(i) * 64);
            ldg_stream(x + 8, chunk0 + static_cast<int64_t>(i) * 64 + 32);
        } else {  // an end of the row, or past this CTA's part
            const int first = 32 * i - off;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int e = first + 2 * j;
                const uint32_t lo = i < c1 && e >= 0 && e < a.V ? row[e] : 0xFC00u, hi = i < c1 && e + 1 >= 0 && e + 1 < a.V ? row[e + 1] : 0xFC00u;
                x[j] = lo | hi << 16;
            }
        }
    };
    griddep_wait();
    int base = c0 + warp * 32;
    if (base < c1) load(base + lane);
    float temp = a.temperature ? a.temperature[m] : 1.f;
    if (!(temp > 0.f)) temp = 1.f;
    const float factor = fminf(1.44269504088896341f / temp, 1e30f);
    const Scale c = {factor, factor > 16.f};

    int tchunk[kG];
    uint32_t gt[kG], ge[kG], above[kG];
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        const int tok = j < a.given ? a.tokens[static_cast<int64_t>(m) * a.given + j] : -1;
        const bool there = tok >= 0 && tok < a.V;
        const uint32_t bits = there ? row[tok] : 0x7C00u;
        gt[j] = bits * 0x10001u;
        ge[j] = below(bits) * 0x10001u;
        tchunk[j] = there ? (tok + off) / 32 : 0;
        above[j] = 0;
        if (rank == 0 && warp == j % kWarps) {  // equal ones before it in its own chunk, which the counts leave out
            const int e = 32 * tchunk[j] - off + lane;
            const bool equal = there && e >= 0 && e < tok && key_of(row[e]) == key_of(bits);
            const uint32_t n = __popc(__ballot_sync(0xffffffffu, equal));
            if (lane == 0) sh.given[j] = bits | n << 16;
        }
    }

    Sums run = {-INFINITY, 0.f, 0.f};
    float best = -INFINITY;  // of this thread's chunks, and the first that has it
    int best_chunk = -1;
    const unsigned long long c2 = pack_f2(factor, factor);
    const uint32_t slot = smem_u32(sh.next[warp]);
    bool copied = false;  // this step's chunks
    for (; base < c1; base += kThreads) {
        const int i = base + lane, after = base + kThreads;
        if (copied) {  // a lane's 16-byte units in an order of its own: 8 lanes, 8 places in the banks
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 v = lds128(slot + 64u * lane + 16u * (q ^ (lane >> 1 & 3)));
                x[4 * q] = v.x;
                x[4 * q + 1] = v.y;
                x[4 * q + 2] = v.z;
                x[4 * q + 3] = v.w;
            }
            __syncwarp();
        } else if (base != c0 + warp * 32) {
            load(i);
        }
        copied = after >= inner0 && after + 32 <= min(c1, inner1) && in_bounds(m * a.stride + 32LL * (after + 32) - off <= total, status);
        if (copied) {
            const unsigned char* from = chunk0 + static_cast<int64_t>(after) * 64 + 16 * lane;
#pragma unroll
            for (int q = 0; q < 4; ++q) copy16(slot + 512u * q + 16u * lane, from + 512 * q);
        }
        uint32_t hi = max2(x[0], x[1]);
#pragma unroll
        for (int j = 2; j < 16; ++j) hi = max2(hi, x[j]);
        hi = max2(hi, kMasked2);  // (NaN alone)
        hi = max2(hi, __byte_perm(hi, hi, 0x1032));
        if (TOP && i < c1) chunk_max[i - c0] = static_cast<uint16_t>(hi & 0xFFFFu);
        const __half2 hi2 = *reinterpret_cast<const __half2*>(&hi);
        const float most = __low2float(hi2);
        if (TOP && most > best) {
            best = most;
            best_chunk = i - c0;
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const uint32_t t = i < tchunk[j] ? ge[j] : gt[j];
            const __half2 t2 = *reinterpret_cast<const __half2*>(&t);
            if (__any_sync(0xffffffffu, most > __low2float(t2))) {
                uint32_t n = 0;  // -1 for a logit above, in 16 bits: -2^16 hi + (2^16 - 1) lo
#pragma unroll
                for (int q = 0; q < 16; q += 2)
                    n += __hgt2_mask(*reinterpret_cast<const __half2*>(&x[q]), t2) + __hgt2_mask(*reinterpret_cast<const __half2*>(&x[q + 1]), t2);
                const int lo = static_cast<int>((0u - n) & 0xFFFFu);
                above[j] += static_cast<uint32_t>(2 * lo - (static_cast<int>(n + lo) >> 16));
            }
        }
        if (most > run.m) rescale(run, most, c);
        if (run.m < INFINITY && (run.m + 65504.f) * factor > 160.f) {
            unsigned long long s = pack_f2(0.f, 0.f), d = s;
            const float k = c.far ? run.m : __fmul_rn(run.m, factor);
            const unsigned long long less = pack_f2(-k, -k);
            auto add = [&](auto far) {
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const uint32_t v = max2(x[q], 0xFBFFFBFFu);  // (-65504, -65504)
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
                    const unsigned long long l = pack_f2(f.x, f.y), e = decltype(far)::value ? mul_f2(add_f2(l, less), c2) : fma_f2(l, c2, less);
                    float e0, e1;
                    unpack_f2(e, e0, e1);
                    const unsigned long long w = pack_f2(ex2(e0), ex2(e1));
                    s = add_f2(s, w);
                    d = fma_f2(w, e, d);
                }
            };
            if (c.far)
                add(std::true_type());
            else
                add(std::false_type());
            float p, q;
            unpack_f2(s, p, q);
            run.s += p + q;
            unpack_f2(d, p, q);
            run.d += p + q;
        } else if (run.m > -INFINITY) {
#pragma unroll
            for (int q = 0; q < 32; ++q) {
                const uint32_t w = q & 1 ? x[q >> 1] >> 16 : x[q >> 1] & 0xFFFFu;
                const float l = __half2float(__ushort_as_half(static_cast<unsigned short>(w)));
                const float e = run.m == INFINITY ? (l == run.m ? 0.f : -200.f) : c.from(l, run.m);
                const float y = l > -INFINITY ? ex2(e) : 0.f;
                run.s += y;
                run.d = y > 0.f ? fmaf(y, e, run.d) : run.d;
            }
        }
    }

    // ---- the CTA's sums and counts
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) run = joined(run, shuffled(run, o), c);
    if (lane == 0) sh.part[warp] = run;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        const uint32_t n = __reduce_add_sync(0xffffffffu, above[j]);
        if (lane == 0) sh.above[warp][j] = n;
    }
    const int n = a.top, chunks = c1 - c0;
    uint32_t mine = 0;
    if (TOP) {
        auto key_with = [](uint32_t bits, int i) {  // 0 for a chunk of masked logits
            const uint32_t k = key_of(bits);
            return k == 0 ? 0u : k << 16 | (0xFFFFu - static_cast<uint32_t>(i));
        };
        mine = best_chunk < 0 ? 0u : key_with(__half_as_ushort(__float2half_rn(best)), best_chunk);
        sh.first[threadIdx.x] = mine;
        for (int i = chunks + threadIdx.x; i < (chunks + 7) / 8 * 8; i += kThreads) chunk_max[i] = 0xFC00u;
        if (threadIdx.x == 0) {
            sh.count = sh.found = 0;
            sh.least = 1;
        }
        if (threadIdx.x < kMaxTop) sh.best[threadIdx.x] = 0;
    }
    __syncthreads();
    if (warp == 0) {
        run = lane < kWarps ? sh.part[lane] : Sums{-INFINITY, 0.f, 0.f};
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) run = joined(run, shuffled(run, o), c);
        if (lane == 0) sh.whole = run;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const uint32_t all = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.above[lane][j] : 0u);
            if (lane == 0) sh.above_whole[j] = all;
        }
    }

    if (TOP) {
        auto key_with = [](uint32_t bits, int i) {
            const uint32_t k = key_of(bits);
            return k == 0 ? 0u : k << 16 | (0xFFFFu - static_cast<uint32_t>(i));
        };
        // A lower bound of the n-th largest maximum: the n-th largest of the threads'. Few maxima are above it.
        if (mine != 0) {
            int before = 0;
#pragma unroll 8
            for (int i = 0; i < kThreads; i += 4) {
                const uint4 q = *reinterpret_cast<const uint4*>(sh.first + i);
                before += (q.x > mine) + (q.y > mine) + (q.z > mine) + (q.w > mine);
            }
            if (before == n - 1) sh.least = mine;
        }
        __syncthreads();
        uint32_t least = sh.least;
        int found;
        for (;;) {  // (once, but for rows made to have hundreds of maxima above the bound)
            const __half2 bound = __half2half2(__float2half_rn(value_of(max(least >> 16, 0x0400u))));  // (at the lowest: all finite ones)
            for (int i = 8 * threadIdx.x; i < chunks; i += 8 * kThreads) {
                const uint4 q = *reinterpret_cast<const uint4*>(chunk_max + i);
                const uint32_t h[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (__hbeq2(__hge2(*reinterpret_cast<const __half2*>(&h[j]), bound), __float2half2_rn(0.f))) continue;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t k = key_with(e ? h[j] >> 16 : h[j] & 0xFFFFu, i + 2 * j + e);
                        if (k < least) continue;
                        const int at = atomicAdd(&sh.count, 1);
                        if (at < kCandidates) sh.keys[at] = k;
                    }
                }
            }
            __syncthreads();
            found = min(sh.count, kCandidates);
            const bool more = sh.count > kCandidates;
            for (int i = threadIdx.x; i < found; i += kThreads) {
                const uint32_t k = sh.keys[i];
                int place = 0;
#pragma unroll 8
                for (int j = 0; j < found; ++j) place += sh.keys[j] > k;
                if (place < n) sh.chunk[place] = 0xFFFFu - (k & 0xFFFFu);
                if (place == min(n, found) - 1) sh.last = more ? k : k >> 16;
            }
            __syncthreads();
            if (!more) break;
            least = sh.last;  // at least n of the maxima in the list: the others go
            if (threadIdx.x == 0) sh.count = 0;
            __syncthreads();
        }
        const int named = min(n, found);
        const uint32_t enough = named == n ? sh.last : 1u;
        for (int i = warp; i < named; i += kWarps) {
            const int el = (c0 + static_cast<int>(sh.chunk[i])) * kChunk - off + lane;
            const bool there = el >= 0 && el < a.V && in_bounds(el < 0 || el >= a.V || m * a.stride + el < total, status);
            const uint32_t k = there ? key_of(row[el]) : 0u;
            if (k >= enough) sh.cand[atomicAdd(&sh.found, 1)] = static_cast<unsigned long long>(k) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(el));
        }
        __syncthreads();
        found = sh.found;
        for (int i = threadIdx.x; i < found; i += kThreads) {
            const unsigned long long k = sh.cand[i];
            int place = 0;
#pragma unroll 8
            for (int j = 0; j < found; ++j) place += sh.cand[j] > k;
            if (place < n) sh.best[place] = k;
        }
    }

    if (C > 1) {
        cluster_sync_all();
        if (rank == 0) {
            if (TOP) {  // every CTA's first tokens in order: a place is what all of them have above
                for (int i = threadIdx.x; i < C * n; i += kThreads) {
                    const uint32_t at = map_peer(smem_u32(&sh.best[i % n]), static_cast<uint32_t>(i / n));
                    unsigned long long k;
                    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(k) : "r"(at) : "memory");
                    sh.cand[i] = k;
                }
                __syncthreads();
                if (threadIdx.x < kMaxTop) sh.best[threadIdx.x] = 0;
                __syncthreads();
                for (int i = threadIdx.x; i < C * n; i += kThreads) {
                    const unsigned long long k = sh.cand[i];
                    int place = 0;
#pragma unroll 4
                    for (int p = 0; p < C; ++p) place += above_in(sh.cand + p * n, n, k);
                    if (k != 0 && place < n) sh.best[place] = k;
                }
            }
            if (warp == 0) {
                run = {-INFINITY, 0.f, 0.f};
                if (lane < C) {
                    const uint32_t at = map_peer(smem_u32(&sh.whole), static_cast<uint32_t>(lane));
                    run = {ld_dsmem_f1(at), ld_dsmem_f1(at + 4), ld_dsmem_f1(at + 8)};
                }
                uint32_t counts[kG];
#pragma unroll
                for (int j = 0; j < NG; ++j)
                    counts[j] = lane < C ? __float_as_uint(ld_dsmem_f1(map_peer(smem_u32(&sh.above_whole[j]), static_cast<uint32_t>(lane)))) : 0u;
                __syncwarp();  // (every lane has read before rank 0's own are replaced)
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) run = joined(run, shuffled(run, o), c);
                if (lane == 0) sh.whole = run;
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    const uint32_t all = __reduce_add_sync(0xffffffffu, counts[j]);
                    if (lane == 0) sh.above_whole[j] = all;
                }
            }
        }
        cluster_sync_all();
        if (rank != 0) return;
    }
    __syncthreads();

    const Sums all = sh.whole;
    const bool exact = c.far || !(fabsf(all.m) < INFINITY);
    const float log_k = logf(all.s);  // (s = 0: nothing but masked logits)
    const float log_s = exact ? log_k : log_k - 0.693147180559945309f * fmaf(all.m, factor, -__fmul_rn(all.m, factor));
    auto logprob = [&](float l) {
        if (!(l > -INFINITY) || (all.m == INFINITY && l != all.m)) return -INFINITY;  // (whatever the temperature)
        return (l == all.m ? 0.f : __fdiv_rn(l - all.m, temp)) - log_s;
    };
    if (threadIdx.x == 0 && a.entropy) a.entropy[m] = all.s > 0.f ? log_k - all.d * 0.693147180559945309f / all.s : 0.f;
    if (static_cast<int>(threadIdx.x) < NG && static_cast<int>(threadIdx.x) < a.given) {
        const int64_t at = static_cast<int64_t>(m) * a.given + threadIdx.x;
        const int t = a.tokens[at];
        float lp = 0.f;
        int place = 0;
        if (t >= 0 && t < a.V) {
            const uint32_t bits = sh.given[threadIdx.x] & 0xFFFFu;
            lp = logprob(__half2float(__ushort_as_half(static_cast<unsigned short>(bits))));
            if (key_of(bits) != 0) place = 1 + static_cast<int>(sh.above_whole[threadIdx.x] + (sh.given[threadIdx.x] >> 16));
        } else if (t >= a.V) {
            record_error(status, kErrBounds);
        }
        if (a.logprob) a.logprob[at] = lp;
        if (a.rank) a.rank[at] = place;
    }
    if (TOP && static_cast<int>(threadIdx.x) < a.top) {
        const int64_t at = static_cast<int64_t>(m) * a.top + threadIdx.x;
        const unsigned long long k = sh.best[threadIdx.x];
        a.top_tokens[at] = k == 0 ? -1 : static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k));
        a.top_logprob[at] = k == 0 ? -INFINITY : logprob(value_of(static_cast<uint32_t>(k >> 32)));
    }
}

template <int NG, int kThreads>
cudaError_t launch_with(const LogprobArgs& a, int M, int C, cudaStream_t s, unsigned* status) {
    const bool top = a.top > 0;
    auto kern = top ? logprobs_kernel<NG, true, kThreads> : logprobs_kernel<NG, false, kThreads>;
    const int chunks = ((a.V + 31 + 31) / 32 + C - 1) / C;
    const size_t smem = top ? (static_cast<size_t>(chunks) * 2 + 31) / 16 * 16 : 0;
    if (top) {  // the most that a call can need: another thread's call may be between here and its launch
        constexpr int most = ((1000000 + 62) / 32 * 2 + 31) / 16 * 16;
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(C) * static_cast<unsigned>(M), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
    if (C > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(C);
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    const int64_t total = static_cast<int64_t>(M - 1) * a.stride + a.V;
    return cudaLaunchKernelEx(&cfg, kern, a, C, total, status);
}

template <int NG>
cudaError_t launch_ng(const LogprobArgs& a, int M, int C, bool wide, cudaStream_t s, unsigned* status) {
    return wide ? launch_with<NG, 256>(a, M, C, s, status) : launch_with<NG, 128>(a, M, C, s, status);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams& p, int sm_count, cudaStream_t s, unsigned* status) {
    const LogprobArgs a = {p.logits, p.stride, p.V, p.tokens, p.given, p.top, p.temperature, p.logprob, p.rank, p.entropy, p.top_tokens, p.top_logprob};
    // Few rows: CTAs until every SM has two, each with 4096 logits at least; many: as many as even out the waves.
    int C = 1;
    while (C < 8 && static_cast<int64_t>(p.M) * C * 2 <= 2 * sm_count && p.V / (2 * C) >= 4096) C *= 2;
    const bool wide = p.M < 4 * sm_count;
    if (p.given <= 0) return launch_ng<0>(a, p.M, C, wide, s, status);
    if (p.given <= 1) return launch_ng<1>(a, p.M, C, wide, s, status);
    if (p.given <= 2) return launch_ng<2>(a, p.M, C, wide, s, status);
    if (p.given <= 4) return launch_ng<4>(a, p.M, C, wide, s, status);
    return launch_ng<8>(a, p.M, C, wide, s, status);
}

}  // namespace w4a16
