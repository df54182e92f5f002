// Token sampling: temperature, top-k, top-p and min-p from a given uniform number per row, without a sort.
//
//   order   logits descending, ties by lower index (NaN and -inf: masked, never chosen)
//   weight  W = rne(2^40 w), w = exp((l - l_max) / T) in binary32, w = 1 where l = l_max
//   kept    the first k; of those, each whose preceding mass is below p times their mass; w >= min_p;
//           the first one always
//   token   the first kept one at which the running mass exceeds u times the kept mass
//
// Weights are whole numbers, so every mass is an exact 64-bit sum: the result does not depend on the
// order of additions, and repeats are identical. fp16 logits have at most 65,536 values and equal logits
// have equal weights, so a row is described by how often each value occurs: a thread-block cluster per
// row counts its values in shared memory (one pass over the logits, one atomic each; 16-bit counters,
// each CTA's slice is below 65,536 elements), folds the counts into 2048 coarse bins of count and mass,
// and every decision above is then a search in the 2048 prefix sums followed by a look at the 32
// values of one bin. Only the chosen value's position is looked up in the logits again.
#include "common.cuh"
#include "internal.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 512;
constexpr int kBins = 2048;           // coarse bins of 32 adjacent values
constexpr uint32_t kMaskedKey = 0x03FFu;  // -inf; every finite value's key is above
constexpr size_t kHistBytes = 65536 * 2;
constexpr size_t kSmemBytes = kHistBytes + 2 * kBins * (4 + 8) + 1024;

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
__device__ __forceinline__ unsigned long long ld_dsmem_u64(uint32_t addr) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_dsmem_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
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

__device__ __forceinline__ Fine fine_of(int bin, uint32_t hist, int C, uint32_t cnt0, unsigned long long mass0,
                                        const Softmax& sm) {
    const int lane = threadIdx.x & 31;
    Fine f;
    f.key = static_cast<uint32_t>(bin * 32 + 31 - lane);
    f.count = 0;
    for (int r = 0; r < C; ++r) f.count += ld_dsmem_u16(map_peer(hist + f.key * 2, r));
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
                  int32_t* __restrict__ tokens, float* __restrict__ probs, int C) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    uint32_t* hist = reinterpret_cast<uint32_t*>(smem + 1024);  // two 16-bit counters a word
    unsigned long long* bin_mass = reinterpret_cast<unsigned long long*>(smem + 1024 + kHistBytes);
    unsigned long long* all_mass = bin_mass + kBins;
    uint32_t* bin_count = reinterpret_cast<uint32_t*>(all_mass + kBins);
    uint32_t* all_count = bin_count + kBins;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_ctarank();
    const int64_t row = blockIdx.x / C;

    griddep_launch_dependents();
    for (int i = tid; i < static_cast<int>(kHistBytes / 16); i += kThreads)
        reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    griddep_wait();

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
    for (int i = tid; i < vectors; i += kThreads) {
        const uint4 v = *reinterpret_cast<const uint4*>(src + first + 8 * i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            take(w[j] & 0xFFFFu);
            take(w[j] >> 16);
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
    sm.temp = greedy ? 1.f : t;

    // ---- this CTA's counts and masses of the coarse bins
    for (int b = tid; b < kBins; b += kThreads) {
        uint32_t count = 0;
        unsigned long long mass = 0;
        if (b * 32 <= static_cast<int>(kmax)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = (i + (lane >> 1)) & 3;
                const uint4 v = reinterpret_cast<const uint4*>(hist)[b * 4 + at];
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t c = (j & 1) ? w[j / 2] >> 16 : w[j / 2] & 0xFFFFu;
                    if (c != 0) {
                        count += c;
                        mass += c * sm.fixed(static_cast<uint32_t>(b * 32 + at * 8 + j));
                    }
                }
            }
        }
        bin_count[b] = count;
        bin_mass[b] = mass;
    }
    cluster_sync_all();
    // ---- each CTA adds up its share of the bins over the cluster, into rank 0's totals
    const int share = kBins / C;
    for (int i = tid; i < share; i += kThreads) {
        const int b = static_cast<int>(rank) * share + i;
        uint32_t count = 0;
        unsigned long long mass = 0;
        for (int r = 0; r < C; ++r) {
            count += ld_dsmem_u32(map_peer(smem_u32(bin_count + b), r));
            mass += ld_dsmem_u64(map_peer(smem_u32(bin_mass + b), r));
        }
        st_dsmem_u32(map_peer(smem_u32(all_count + b), 0), count);
        st_dsmem_u64(map_peer(smem_u32(all_mass + b), 0), mass);
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
#pragma unroll
        for (int i = 0; i < kPer; ++i) {  // reuse this CTA's own bins, in position order
            bin_count[tid * kPer + i] = cb;
            bin_mass[tid * kPer + i] = mb;
            cb += c[i];
            mb += m[i];
        }
        __syncthreads();
        if (warp == 0) {
            const uint32_t h = smem_u32(hist);
            // last position whose preceding count / mass is <= x
            auto find = [&](auto* before, unsigned long long x) {
                int lo = 0, hi = kBins - 1;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (before[mid] <= x) lo = mid;
                    else hi = mid - 1;
                }
                return lo;
            };
            auto at = [&](int pos) { return fine_of(kBins - 1 - pos, h, C, bin_count[pos], bin_mass[pos], sm); };
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
                    // smallest value with weight >= min_p: a search over the keys, 32 at a time
                    uint32_t base = 0, width = 65536;
                    while (width > 1) {
                        const uint32_t step = max(1u, width / 32);
                        const uint32_t key = min(base + (lane + 1) * step - 1, kmax);
                        const bool yes = key > kMaskedKey && sm.weight(key) >= mp;
                        const int l = __ffs(__ballot_sync(0xffffffffu, yes)) - 1;
                        base += l * step;
                        width = step;
                    }
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
                uint32_t here = lane < C ? ld_dsmem_u16(map_peer(h + key * 2, lane)) : 0, upto = here;
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
    const uint32_t key = sh.pick_key, index = sh.pick_index;
    const int per_warp = ((end - begin + kThreads / 32 - 1) / (kThreads / 32) + 31) / 32 * 32;
    const int w0 = min(end, begin + warp * per_warp), w1 = min(end, w0 + per_warp);
    uint32_t count = 0;
    for (int i = w0 + lane; i < w1; i += 32) count += key_of(src[i]) == key;
    count = __reduce_add_sync(0xffffffffu, count);
    __syncthreads();
    if (lane == 0) sh.warp_count[warp] = count;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < warp; ++i) before += sh.warp_count[i];
    if (index < before || index >= before + count) return;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t hit = __ballot_sync(0xffffffffu, i < w1 && key_of(src[min(i, end - 1)]) == key);
        const uint32_t n = __popc(hit);
        if (index < before + n) {
            if (lane == 0) tokens[row] = i0 + static_cast<int>(__fns(hit, 0, static_cast<int>(index - before) + 1));
            return;
        }
        before += n;
    }
}

}  // namespace

cudaError_t launch_sample(const SampleParams& p, cudaStream_t s, unsigned* status) {
    (void)status;
    // CTAs per row: enough that each counts fewer than 65,536 values; a row alone on the GPU is spread
    // over up to 16.
    int C = 4;
    if (p.M <= 18) C = 8;
    if (p.M <= 9) C = 16;
    while (C < 16 && (p.V + C - 1) / C > 65528) C *= 2;
    const int slice = ((p.V + C - 1) / C + 7) / 8 * 8;
    cudaError_t e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kSmemBytes));
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(p.M) * C), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
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
    return cudaLaunchKernelEx(&cfg, sample_kernel, p.logits, p.stride, p.V, slice, p.temperature, p.top_k, p.top_p,
                              p.min_p, p.u, p.tokens, p.probs, C);
}

}  // namespace w4a16
