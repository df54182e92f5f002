// Log probabilities of rows of fp16 logits, in one pass over a row:
//
//   p_i = exp((l_i - l_max) / T) / S,  S = sum_i exp((l_i - l_max) / T)      (NaN and -inf: p = 0)
//   log p of given tokens, and their places in the order (logits descending, ties by lower index)
//   entropy  -sum p log p = log S - (1 / S) sum_i w_i d_i,  d_i = (l_i - l_max) / T, w_i = exp(d_i): two sums
//            of one sign, nothing cancels
//   the first n of the order
//
// A thread keeps the largest logit so far, S and sum w d relative to it, and rescales both when a larger
// one turns up. A place is a count: logits above the given one, and equal ones before it; "equal or above"
// is "above the next smaller fp16 number", so either is one packed comparison.
//
// The first n: each 32 neighbours (a chunk, four lanes' vectors) leave their maximum in shared memory. The
// first n of a row lie in the n chunks that come first in the order (maximum, then lower chunk): a chunk
// before another has an element before each of the other's. So a search among the maxima names n chunks,
// and only their n * 32 elements are read a second time.
//
// A row is a CTA or a cluster, whose parts rank 0 brings together in a fixed order.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 32;       // elements: 4 vectors of 8
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

template <int NG>
struct __align__(16) Shared {
    unsigned long long best[kMaxTop];          // this CTA's first tokens
    unsigned long long cand[kCandidates];      // (value key, ~index)
    uint32_t keys[kCandidates];                // (value key of a chunk's maximum, ~chunk)
    uint32_t group[32];
    uint32_t chunk[kMaxTop];
    uint32_t last;                             // value key of the n-th chunk
    int count;
    Sums part[kWarps];
    uint32_t above[kWarps][NG == 0 ? 1 : NG];
    Sums whole;                                // of this CTA
    uint32_t above_whole[NG == 0 ? 1 : NG];
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

__device__ __forceinline__ uint4 ldg_stream(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ unsigned long long pack(float lo, float hi) {
    unsigned long long v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ void unpack(unsigned long long v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// `a` seen from the larger maximum m.
__device__ __forceinline__ void rescale(Sums& a, float m, float c) {
    if (a.s == 0.f) {
        a.d = 0.f;
    } else if (m == INFINITY) {
        if (a.m != m) a.s = a.d = 0.f;
    } else {
        const float x = (a.m - m) * c, e = ex2(x);
        a.d = e == 0.f ? 0.f : e * fmaf(x, a.s, a.d);
        a.s *= e;
    }
    a.m = m;
}
__device__ __forceinline__ Sums joined(Sums a, Sums b, float c) {
    const float m = fmaxf(a.m, b.m);
    rescale(a, m, c);
    rescale(b, m, c);
    return {m, a.s + b.s, a.d + b.d};
}

template <int NG, bool TOP>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobArgs a, int C, int64_t total, unsigned* status) {
    extern __shared__ uint16_t chunk_max[];  // fp16 maxima of this CTA's chunks
    __shared__ Shared<NG> sh;
    griddep_launch_dependents();
    const int rank = static_cast<int>(blockIdx.x) % C, m = static_cast<int>(blockIdx.x) / C;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint16_t* row = a.logits + static_cast<int64_t>(m) * a.stride;
    // Vectors are the 16-byte aligned ones that cover the row: vector v holds elements 8 v - off and on.
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) >> 1) & 7u);
    const uint4* vec = reinterpret_cast<const uint4*>(row - off);
    const int NV = (off + a.V + 7) / 8;
    const int per = ((NV + 3) / 4 + C - 1) / C * 4;
    const int v0 = min(NV, rank * per), v1 = min(NV, v0 + per);
    griddep_wait();
    float temp = a.temperature ? a.temperature[m] : 1.f;
    if (!(temp > 0.f)) temp = 1.f;
    const float c = fminf(1.44269504088896341f / temp, 1e30f);

    int tok[NG == 0 ? 1 : NG], tvec[NG == 0 ? 1 : NG];
    uint32_t gt[NG == 0 ? 1 : NG], ge[NG == 0 ? 1 : NG];
    uint32_t above[NG == 0 ? 1 : NG];
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        tok[j] = j < a.given ? a.tokens[static_cast<int64_t>(m) * a.given + j] : -1;
        const bool there = tok[j] >= 0 && tok[j] < a.V;
        const uint32_t bits = there ? row[tok[j]] : 0x7C00u;
        gt[j] = bits * 0x10001u;
        ge[j] = below(bits) * 0x10001u;
        tvec[j] = there ? (tok[j] + off) / 8 : 0;
        above[j] = 0;
    }

    Sums run = {-INFINITY, 0.f, 0.f};
    const unsigned long long c2 = pack(c, c);
    for (int base = v0 + warp * 128; base < v1; base += kWarps * 128) {
        uint32_t x[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int v = base + u * 32 + lane;
            uint4 q = make_uint4(kMasked2, kMasked2, kMasked2, kMasked2);
            const int first = 8 * v - off;
            if (v < v1) {
                if (first >= 0 && first + 8 <= a.V) {
                    if (in_bounds(m * a.stride + first + 8 <= total, status)) q = ldg_stream(vec + v);
                } else {  // the vectors at the ends of the row: only what is inside
                    uint32_t e[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) e[i] = first + i >= 0 && first + i < a.V ? row[first + i] : 0xFC00u;
                    q = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
                }
            }
            x[u][0] = q.x;
            x[u][1] = q.y;
            x[u][2] = q.z;
            x[u][3] = q.w;
        }
        uint32_t hi = kMasked2;
        bool plain[4], all_plain = true;  // no masked logit in the vector
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            uint32_t h = max2(max2(x[u][0], x[u][1]), max2(x[u][2], x[u][3]));
            const uint32_t lo = min2_nan(min2_nan(x[u][0], x[u][1]), min2_nan(x[u][2], x[u][3]));
            const __half2 lo2 = *reinterpret_cast<const __half2*>(&lo);
            plain[u] = __low2float(lo2) > -INFINITY && __high2float(lo2) > -INFINITY;
            all_plain = all_plain && plain[u];
            hi = max2(hi, h);
            if (TOP) {
                h = max2(h, kMasked2);  // (a chunk of NaN alone)
                h = max2(h, __byte_perm(h, h, 0x1032));
                h = max2(h, __shfl_xor_sync(0xffffffffu, h, 1));
                h = max2(h, __shfl_xor_sync(0xffffffffu, h, 2));
                const int v = base + u * 32 + lane;
                if ((lane & 3) == 0 && v < v1) chunk_max[(v - v0) >> 2] = static_cast<uint16_t>(h & 0xFFFFu);
            }
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            __half2 n = __float2half2_rn(0.f);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t t = base + u * 32 + lane < tvec[j] ? ge[j] : gt[j];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    n = __hadd2(n, __hgt2(*reinterpret_cast<const __half2*>(&x[u][i]), *reinterpret_cast<const __half2*>(&t)));
            }
            above[j] += static_cast<uint32_t>(__low2float(n) + __high2float(n));
        }
        const __half2 hi2 = *reinterpret_cast<const __half2*>(&hi);
        const float most = fmaxf(__low2float(hi2), __high2float(hi2));
        if (most > run.m) rescale(run, most, c);
        unsigned long long s = pack(0.f, 0.f), d = s;
        const unsigned long long nm = pack(-run.m, -run.m);
        auto plain_vector = [&](const uint32_t (&v)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
                const unsigned long long e = mul2(add2(pack(f.x, f.y), nm), c2);
                float e0, e1;
                unpack(e, e0, e1);
                const unsigned long long w = pack(ex2(e0), ex2(e1));
                s = add2(s, w);
                d = fma2(w, e, d);
            }
        };
        if (all_plain && run.m < INFINITY) {
#pragma unroll
            for (int u = 0; u < 4; ++u) plain_vector(x[u]);
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (base + u * 32 + lane >= v1) continue;
                if (plain[u] && run.m < INFINITY) {
                    plain_vector(x[u]);
                    continue;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {  // masked or infinite logits among them
                    const uint32_t w = i & 1 ? x[u][i >> 1] >> 16 : x[u][i >> 1] & 0xFFFFu;
                    const float l = __half2float(__ushort_as_half(static_cast<unsigned short>(w)));
                    if (!(l > -INFINITY)) continue;
                    const float e = run.m == INFINITY ? (l == run.m ? 0.f : -200.f) : (l - run.m) * c, y = ex2(e);
                    run.s += y;
                    run.d = y > 0.f ? fmaf(y, e, run.d) : run.d;
                }
            }
        }
        float p, q;
        unpack(s, p, q);
        run.s += p + q;
        unpack(d, p, q);
        run.d += p + q;
    }

    // ---- the CTA's sums and counts, then the cluster's, in a fixed order
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Sums b = {__shfl_xor_sync(0xffffffffu, run.m, o), __shfl_xor_sync(0xffffffffu, run.s, o), __shfl_xor_sync(0xffffffffu, run.d, o)};
        run = joined(run, b, c);
    }
    if (lane == 0) sh.part[warp] = run;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        const uint32_t n = __reduce_add_sync(0xffffffffu, above[j]);
        if (lane == 0) sh.above[warp][j] = n;
    }
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    if (threadIdx.x == 0) {
        Sums all = sh.part[0];
        for (int w = 1; w < kWarps; ++w) all = joined(all, sh.part[w], c);
        sh.whole = all;
    }
    if (threadIdx.x < NG) {
        uint32_t n = 0;
        for (int w = 0; w < kWarps; ++w) n += sh.above[w][threadIdx.x];
        sh.above_whole[threadIdx.x] = n;
    }

    if (TOP) {
        const int n = a.top, chunks = (v1 - v0 + 3) / 4;
        auto chunk_key = [&](int i) {  // 0 for a chunk of masked logits
            const uint32_t k = key_of(chunk_max[i]);
            return k == 0 ? 0u : k << 16 | (0xFFFFu - static_cast<uint32_t>(i));
        };
        // A lower bound of the n-th largest maximum: the n-th largest of 32 groups'. Few maxima are above it.
        uint32_t g = 0;
        for (int i = threadIdx.x; i < chunks; i += kThreads) g = max(g, chunk_key(i));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) g = max(g, __shfl_xor_sync(0xffffffffu, g, o));
        if ((threadIdx.x & 7) == 0) sh.group[threadIdx.x >> 3] = g;
        __syncthreads();
        g = sh.group[lane];
        int before = 0;
        for (int o = 1; o < 32; ++o) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, g, o);
            before += other > g || (other == g && (lane ^ o) < lane);  // (only empty groups are equal)
        }
        uint32_t least = max(1u, __reduce_min_sync(0xffffffffu, before < n ? g : 0xFFFFFFFFu));
        for (;;) {  // (once, but for rows made to have hundreds of maxima above the bound)
            for (int i = threadIdx.x; i < chunks; i += kThreads) {
                const uint32_t k = chunk_key(i);
                if (k >= least) {
                    const int at = atomicAdd(&sh.count, 1);
                    if (at < kCandidates) sh.keys[at] = k;
                }
            }
            __syncthreads();
            const int found = min(sh.count, kCandidates);
            const bool more = sh.count > kCandidates;
            for (int i = threadIdx.x; i < found; i += kThreads) {
                const uint32_t k = sh.keys[i];
                int place = 0;
                for (int j = 0; j < found; ++j) place += sh.keys[j] > k;
                if (place < n) sh.chunk[place] = 0xFFFFu - (k & 0xFFFFu);
                if (place == min(n, found) - 1) sh.last = more ? k : k >> 16;
            }
            __syncthreads();
            if (!more) break;
            least = sh.last;  // at least n of the maxima in the list: the others go
            __syncthreads();
            if (threadIdx.x == 0) sh.count = 0;
            __syncthreads();
        }
        const int named = min(n, sh.count);
        const uint32_t enough = named == n ? sh.last : 1u;
        __syncthreads();
        if (threadIdx.x == 0) sh.count = 0;
        if (threadIdx.x < kMaxTop) sh.best[threadIdx.x] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < named * kChunk; i += kThreads) {
            const int el = (v0 + static_cast<int>(sh.chunk[i / kChunk]) * 4) * 8 - off + i % kChunk;
            if (el < 0 || el >= a.V || el >= 8 * v1 - off) continue;
            if (!in_bounds(m * a.stride + el < total, status)) continue;
            const uint32_t k = key_of(row[el]);
            if (k >= enough) sh.cand[atomicAdd(&sh.count, 1)] = static_cast<unsigned long long>(k) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(el));
        }
        __syncthreads();
        const int found = sh.count;
        for (int i = threadIdx.x; i < found; i += kThreads) {
            const unsigned long long k = sh.cand[i];
            int place = 0;
            for (int j = 0; j < found; ++j) place += sh.cand[j] > k;
            if (place < n) sh.best[place] = k;
        }
    }

    if (C > 1) {
        cluster_sync_all();
        if (rank == 0) {
            if (TOP) {  // the others' first tokens: C * top <= 16 * 32 candidates
                const int n = a.top;
                unsigned long long k = 0;
                for (int i = threadIdx.x; i < C * n; i += kThreads) {
                    const uint32_t at = map_peer(smem_u32(&sh.best[i % n]), static_cast<uint32_t>(i / n));
                    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(k) : "r"(at) : "memory");
                    sh.cand[i] = k;
                }
                __syncthreads();
                if (threadIdx.x < kMaxTop) sh.best[threadIdx.x] = 0;
                __syncthreads();
                for (int i = threadIdx.x; i < C * n; i += kThreads) {
                    k = sh.cand[i];
                    int place = 0;
                    for (int j = 0; j < C * n; ++j) place += sh.cand[j] > k;
                    if (k != 0 && place < n) sh.best[place] = k;
                }
            }
            if (threadIdx.x == 0) {
                Sums all = sh.whole;
                for (int p = 1; p < C; ++p) {
                    const uint32_t at = map_peer(smem_u32(&sh.whole), static_cast<uint32_t>(p));
                    all = joined(all, {ld_dsmem_f1(at), ld_dsmem_f1(at + 4), ld_dsmem_f1(at + 8)}, c);
                }
                sh.whole = all;
            }
            if (threadIdx.x < NG) {
                uint32_t n = sh.above_whole[threadIdx.x];
                for (int p = 1; p < C; ++p)
                    n += __float_as_uint(ld_dsmem_f1(map_peer(smem_u32(&sh.above_whole[threadIdx.x]), static_cast<uint32_t>(p))));
                sh.above_whole[threadIdx.x] = n;
            }
        }
        cluster_sync_all();
        if (rank != 0) return;
    }
    __syncthreads();

    const Sums all = sh.whole;
    const float log_s = logf(all.s);  // (s = 0: nothing but masked logits)
    auto logprob = [&](float l) {
        if (!(l > -INFINITY) || (all.m == INFINITY && l != all.m)) return -INFINITY;  // (whatever the temperature)
        return (l == all.m ? 0.f : __fdiv_rn(l - all.m, temp)) - log_s;
    };
    if (threadIdx.x == 0 && a.entropy) a.entropy[m] = all.s > 0.f ? log_s - all.d * 0.693147180559945309f / all.s : 0.f;
    if (threadIdx.x < NG && threadIdx.x < a.given) {
        const int64_t at = static_cast<int64_t>(m) * a.given + threadIdx.x;
        const int t = a.tokens[at];
        float lp = 0.f;
        int place = 0;
        if (t >= 0 && t < a.V) {
            const uint32_t bits = row[t], key = key_of(bits);
            lp = logprob(__half2float(__ushort_as_half(static_cast<unsigned short>(bits))));
            if (key != 0) {
                place = 1 + static_cast<int>(sh.above_whole[threadIdx.x]);
                for (int i = max(0, (t + off) / 8 * 8 - off); i < t; ++i) place += key_of(row[i]) == key;  // equal ones in its own vector
            }
        } else if (t >= a.V) {
            record_error(status, kErrBounds);
        }
        if (a.logprob) a.logprob[at] = lp;
        if (a.rank) a.rank[at] = place;
    }
    if (TOP && threadIdx.x < a.top) {
        const int64_t at = static_cast<int64_t>(m) * a.top + threadIdx.x;
        const unsigned long long k = sh.best[threadIdx.x];
        a.top_tokens[at] = k == 0 ? -1 : static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k));
        a.top_logprob[at] = k == 0 ? -INFINITY : logprob(value_of(static_cast<uint32_t>(k >> 32)));
    }
}

template <int NG>
cudaError_t launch_ng(const LogprobArgs& a, int M, int C, cudaStream_t s, unsigned* status) {
    const bool top = a.top > 0;
    auto kern = top ? logprobs_kernel<NG, true> : logprobs_kernel<NG, false>;
    const int chunks = (((a.V + 14) / 8 + 3) / 4 + C - 1) / C;
    const size_t smem = top ? (static_cast<size_t>(chunks) * 2 + 15) / 16 * 16 : 0;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (C > 8) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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

}  // namespace

cudaError_t launch_logprobs(const LogprobParams& p, int sm_count, cudaStream_t s, unsigned* status) {
    const LogprobArgs a = {p.logits, p.stride, p.V, p.tokens, p.given, p.top, p.temperature, p.logprob, p.rank, p.entropy, p.top_tokens, p.top_logprob};
    // Few rows: CTAs until every SM has two, each with 4096 logits at least; many: as many as even out the waves.
    int C = 1;
    while (C < 16 && static_cast<int64_t>(p.M) * C * 2 <= 2 * sm_count && p.V / (2 * C) >= 4096) C *= 2;
    if (p.given <= 0) return launch_ng<0>(a, p.M, C, s, status);
    if (p.given <= 1) return launch_ng<1>(a, p.M, C, s, status);
    if (p.given <= 2) return launch_ng<2>(a, p.M, C, s, status);
    if (p.given <= 4) return launch_ng<4>(a, p.M, C, s, status);
    return launch_ng<8>(a, p.M, C, s, status);
}

}  // namespace w4a16
