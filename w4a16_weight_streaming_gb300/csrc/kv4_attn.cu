// Attention over the 4-bit paged key/value cache for few query rows a sequence (decode and short verify
// steps): o = softmax(scale q k'^T) v', k' and v' the stored values min + code * scale.
//
// Memory-bound: every cached byte is used by the 5 or so query heads of its key/value head, times the
// queries of a verify step. The rows of one key/value head are taken 8 at a time, one column each of an
// m16n8k16 matrix instruction whose 16 rows are cached tokens (scores) or elements (output):
//   scores  S^T[16 tokens][8 rows]   = K codes [16 x D] . Q^T[D x 8]
//   output  O^T[D][8 rows]          += V codes^T [D x 16] . P[16 x 8]
// The codes go into the instruction as they are: a nibble in the low bits of an fp16 is the subnormal
// code * 2^-24, exact, so a pair of operands costs one AND (the nibbles one place up are 16 times that;
// for keys they have an accumulator of their own, for values they are other rows of the output). The
// parameters come in around the products, in fp32, per token t and group y of 64 elements:
//   S_t  = sum_y scale_ty (sum_d q_d code_td) + min_ty (sum_d q_d)
//   O_d  = sum_t (P_t scale_ty) code_td + sum_t P_t min_ty
// P_t scale_ty goes into the instruction as two fp16 numbers, its rounding and what that left over: the
// codes' part and the minimums' part of a value cancel where the value is small, so one rounding of P_t
// scale_ty would be off by 2^-11 of the group's whole range. A power of two keeps both normal.
//
// Work is a list of (sequence, 8 rows, key/value head, 16-token tile); every CTA takes an equal run of
// it, whatever the lengths, and its warps take the run's tiles in turn, each with a running maximum and
// sum of its own, so that no warp waits for another inside a run. A tile is one bulk copy into the
// warp's own ring in shared memory. Runs that end inside a row group leave their part in the workspace;
// the CTA that arrives last there adds the parts in CTA order.
#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace w4a16 {
namespace {

constexpr int kRows = 8;  // query rows of one work unit

template <int D>
struct Decode {
    static constexpr int kWarps = D == 256 ? 12 : 16;
    static constexpr int kStages = D == 256 ? 3 : D == 128 ? 4 : 6;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kTile = Kv4<D>::kTileBytes;
    static constexpr int kRing = kWarps * kStages * kTile;
    static constexpr int kPitch = D + 4;  // floats between rows of a warp's part: conflict-free stores
    static constexpr int kJoin = kWarps * kRows * kPitch * 4;
    static constexpr int kData = kRing > kJoin ? kRing : kJoin;
    static constexpr int kSmem = kData + kWarps * kStages * 8 + kWarps * kRows * 8 + 256;
    static constexpr int kPart = kRows * (D + 2);  // floats of one workspace part: m, l, then rows
};

constexpr int kMaxCtas = 256;
constexpr size_t kCounterBytes = kMaxCtas * 4;

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ float lo_f(uint32_t h2) { return __low2float(*reinterpret_cast<const __half2*>(&h2)); }
__device__ __forceinline__ float hi_f(uint32_t h2) { return __high2float(*reinterpret_cast<const __half2*>(&h2)); }

// The parameters of one token: one (scale, min) pair a group.
template <int G>
__device__ __forceinline__ void lds_params(uint32_t addr, uint32_t (&p)[G]) {
    if constexpr (G == 4) {
        const uint4 v = lds128(addr);
        p[0] = v.x;
        p[1] = v.y;
        p[2] = v.z;
        p[3] = v.w;
    } else if constexpr (G == 2) {
        const uint2 v = lds64(addr);
        p[0] = v.x;
        p[1] = v.y;
    } else {
        p[0] = lds32(addr);
    }
}

struct Seq {
    int q0, q_len, n;  // first row of q, rows, cached tokens
    int row_groups, units, tiles;
    bool bad;
};

__device__ __forceinline__ Seq seq_of(const Kv4AttnParams& p, const Kv4View& c, int b) {
    Seq s;
    const int q0 = p.q_start[b], q1 = p.q_start[b + 1], n = p.kv_len[b];
    s.q0 = min(max(q0, 0), p.M);
    const int end = min(max(q1, s.q0), p.M);
    s.q_len = end - s.q0;
    s.n = min(max(n, 0), p.max_pages << c.page_shift);
    s.bad = s.q0 != q0 || end != q1 || s.n != n;
    const int grp = p.heads / c.kv_heads;
    s.row_groups = (s.q_len * grp + kRows - 1) / kRows;
    s.units = s.row_groups * c.kv_heads;
    s.tiles = max(1, (s.n + kKv4Tile - 1) / kKv4Tile);
    return s;
}

template <int D>
__global__ void __launch_bounds__(Decode<D>::kThreads, 1)
    kv4_decode_kernel(const Kv4AttnParams p, const Kv4View cache, uint64_t timeout_ns, unsigned* status) {
    using C = Decode<D>;
    using T = Kv4<D>;
    constexpr int G = T::kGroups, NW = C::kWarps, S = C::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    float* s_max = reinterpret_cast<float*>(smem + C::kData + NW * S * 8);  // [NW][8]
    float* s_sum = s_max + NW * kRows;
    int64_t* s_plan = reinterpret_cast<int64_t*>(s_sum + NW * kRows);  // run length, offset in the first sequence
    int* s_first = reinterpret_cast<int*>(s_plan + 4);
    int* s_abort = s_first + 1;
    int* s_last = s_first + 2;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * S * C::kTile;
    const uint32_t bars = smem_u32(smem + C::kData) + warp * S * 8;
    const int grp = p.heads / cache.kv_heads;

    if (lane == 0)
        for (int i = 0; i < S; ++i) mbar_init(bars + 8 * i, 1);
    if (tid == 0) *s_abort = 0;
    fence_barrier_init();
    griddep_launch_dependents();
    griddep_wait();

    // ---- this CTA's run of the work list
    if (warp == 0) {
        int64_t total = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            int64_t c = 0;
            if (b0 + lane < p.B) {
                const Seq s = seq_of(p, cache, b0 + lane);
                c = static_cast<int64_t>(s.units) * s.tiles;
                if (s.bad && blockIdx.x == 0) record_error(status, kErrBounds);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
            total += c;
        }
        const int64_t per = max((total + gridDim.x - 1) / gridDim.x, static_cast<int64_t>(NW));
        const int64_t w0 = min(total, per * blockIdx.x), w1 = min(total, w0 + per);
        int64_t at = 0;
        int first = p.B;
        for (int b0 = 0; b0 < p.B && w0 < w1; b0 += 32) {
            int64_t c = 0;
            if (b0 + lane < p.B) {
                const Seq s = seq_of(p, cache, b0 + lane);
                c = static_cast<int64_t>(s.units) * s.tiles;
            }
            int64_t upto = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, at + upto > w0);
            if (hit != 0) {
                const int l = __ffs(hit) - 1;
                first = b0 + l;
                at += __shfl_sync(0xffffffffu, upto - c, l);
                break;
            }
            at += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (lane == 0) {
            s_plan[0] = w1 - w0;
            s_plan[1] = w0 - at;
            s_plan[2] = per;
            s_plan[3] = at;  // work list position of the first sequence
            *s_first = first;
        }
    }
    __syncthreads();
    int64_t left = s_plan[0], off = s_plan[1], seq_at = s_plan[3];
    const int64_t per = s_plan[2];
    uint32_t phase = 0;  // one bit per ring stage

    for (int b = *s_first; left > 0 && b < p.B;) {
        const Seq sq = seq_of(p, cache, b);
        const int64_t cost = static_cast<int64_t>(sq.units) * sq.tiles;
        if (off >= cost) {
            off -= cost;  // a sequence without rows
            seq_at += cost;
            ++b;
            continue;
        }
        const int unit = static_cast<int>(off / sq.tiles);
        const int t0 = static_cast<int>(off - static_cast<int64_t>(unit) * sq.tiles);
        const int t1 = static_cast<int>(min(static_cast<int64_t>(sq.tiles), t0 + left));
        const int kvh = unit / sq.row_groups, rt = unit - kvh * sq.row_groups;
        const int rows = min(kRows, sq.q_len * grp - rt * kRows);
        // tokens that a row sees; rows of this unit beyond the sequence's see as many as the last
        auto seen = [&](int r) {
            const int pos = (rt * kRows + min(r, rows - 1)) / grp;
            return p.causal ? max(0, sq.n - (sq.q_len - 1 - pos)) : sq.n;
        };
        const int lim0 = seen(2 * t), lim1 = seen(2 * t + 1), lim_min = seen(0), lim_max = seen(kRows - 1);
        const int t1e = min(t1, (lim_max + kKv4Tile - 1) / kKv4Tile);
        const int mine = max(0, (t1e - t0 - warp + NW - 1) / NW);  // tiles of this warp: t0 + warp + NW i

        // ---- the ring: page numbers of 32 of the warp's tiles at a time, one bulk copy a tile
        int page_of = -1;
        auto fetch_pages = [&](int i0) {
            const int tile = t0 + warp + NW * (i0 + lane);
            page_of = -1;
            if (tile < t1e) {
                page_of = p.block_table[static_cast<int64_t>(b) * p.max_pages + (tile * kKv4Tile >> cache.page_shift)];
                if (page_of < 0 || page_of >= cache.num_pages) {
                    record_error(status, kErrBounds);
                    page_of = -1;
                }
            }
        };
        uint32_t there = 0;  // tiles in the ring whose page exists, by stage
        auto issue = [&](int i) {
            if ((i & 31) == 0) fetch_pages(i);
            const int page = __shfl_sync(0xffffffffu, page_of, i & 31);
            const int st = i % S;
            const int tile = t0 + warp + NW * i;
            bool ok = page >= 0;
            int64_t from = 0;
            if (ok) {
                from = cache.tile_offset<D>(page, kvh, tile * kKv4Tile & ((1 << cache.page_shift) - 1));
                ok = in_bounds(from >= 0 && from + C::kTile <= cache.bytes<D>(), status);
            }
            there = ok ? there | (1u << st) : there & ~(1u << st);
            if (ok && lane == 0) {
                mbar_arrive_expect_tx(bars + 8 * st, C::kTile);
                bulk_g2s(ring + st * C::kTile, cache.pages + from, C::kTile, bars + 8 * st, policy_evict_first());
            }
        };
        for (int i = 0; i < min(S, mine); ++i) issue(i);

        // ---- Q^T fragments (row g of the unit), and the sums of q over each group for rows 2t, 2t + 1
        uint32_t q[G][2][4];
        float qs0[G], qs1[G];
        {
            const int pos = (rt * kRows + g) / grp, hd = (rt * kRows + g) % grp;
            const uint16_t* src = p.q + (sq.q0 + pos) * p.q_stride + static_cast<int64_t>(kvh * grp + hd) * D;
            const float c1 = p.scale * 1.4426950408889634f;
#pragma unroll
            for (int y = 0; y < G; ++y) {
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (g < rows) v = *reinterpret_cast<const uint4*>(src + y * kKv4Group + 16 * t + 8 * w);
                    q[y][w][0] = v.x;
                    q[y][w][1] = v.y;
                    q[y][w][2] = v.z;
                    q[y][w][3] = v.w;
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum += lo_f(q[y][w][i]) + hi_f(q[y][w][i]);
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                qs0[y] = __shfl_sync(0xffffffffu, sum, 8 * t) * c1;
                qs1[y] = __shfl_sync(0xffffffffu, sum, 8 * t + 4) * c1;
            }
        }
        const float c0 = p.scale * (1.4426950408889634f * 16777216.f);  // scale log2(e) 2^24
        float o[4 * G][4], om[G][2];
#pragma unroll
        for (int i = 0; i < 4 * G; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
        for (int y = 0; y < G; ++y) om[y][0] = om[y][1] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        float vmul = 1.f, vcap = 0.f;  // P scale is taken times vmul = 2^e; scales up to vcap fit

        for (int i = 0; i < mine; ++i) {
            const int st = i % S;
            const bool have = (there >> st) & 1u;
            const uint32_t tile_s = ring + st * C::kTile;
            if (have) {
                if (!warp_spin(bars + 8 * st, (phase >> st) & 1u, s_abort, timeout_ns, status)) {
                    // give up: let the copies in flight land (bounded) before their memory is used again
                    for (int k = 0; k < S; ++k)
                        for (int n = 0; n < 65536 && !mbar_test_wait(bars + 8 * k, (phase >> k) & 1u); ++n) {
                        }
                    break;
                }
                phase ^= 1u << st;
                const int tok = (t0 + warp + NW * i) * kKv4Tile;
                uint32_t kp[2][G], vp[2][G];
                lds_params<G>(tile_s + T::kKParams + g * G * 4, kp[0]);
                lds_params<G>(tile_s + T::kKParams + (g + 8) * G * 4, kp[1]);
                lds_params<G>(tile_s + T::kVParams + g * G * 4, vp[0]);
                lds_params<G>(tile_s + T::kVParams + (g + 8) * G * 4, vp[1]);
                const bool edge = tok + kKv4Tile > lim_min;
                if (edge) {  // memory beyond the cached tokens may hold anything
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (tok + 8 * h + g >= sq.n) {
#pragma unroll
                            for (int y = 0; y < G; ++y) kp[h][y] = vp[h][y] = 0;
                        }
                }
                // scores of tokens g, g + 8 (s[0..1], s[2..3]) and rows 2t, 2t + 1, in powers of two
                float s[4] = {0.f, 0.f, 0.f, 0.f};
                auto group_scores = [&](int y, uint32_t a_w0, uint32_t b_w0, uint32_t a_w1, uint32_t b_w1) {
                    float x[4] = {0.f, 0.f, 0.f, 0.f}, z[4] = {0.f, 0.f, 0.f, 0.f};
                    constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;
                    mma16816(x, a_w0 & kLow, b_w0 & kLow, (a_w0 >> 8) & kLow, (b_w0 >> 8) & kLow, q[y][0][0], q[y][0][2]);
                    mma16816(z, a_w0 & kHigh, b_w0 & kHigh, (a_w0 >> 8) & kHigh, (b_w0 >> 8) & kHigh, q[y][0][1], q[y][0][3]);
                    mma16816(x, a_w1 & kLow, b_w1 & kLow, (a_w1 >> 8) & kLow, (b_w1 >> 8) & kLow, q[y][1][0], q[y][1][2]);
                    mma16816(z, a_w1 & kHigh, b_w1 & kHigh, (a_w1 >> 8) & kHigh, (b_w1 >> 8) & kHigh, q[y][1][1], q[y][1][3]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float sc = lo_f(kp[h][y]) * c0, mn = hi_f(kp[h][y]);
                        s[2 * h] = fmaf(sc, fmaf(z[2 * h], 0.0625f, x[2 * h]), fmaf(mn, qs0[y], s[2 * h]));
                        s[2 * h + 1] = fmaf(sc, fmaf(z[2 * h + 1], 0.0625f, x[2 * h + 1]), fmaf(mn, qs1[y], s[2 * h + 1]));
                    }
                };
                if constexpr (G == 1) {
                    const uint2 a = lds64(tile_s + lane * 8), c = lds64(tile_s + (32 + lane) * 8);
                    group_scores(0, a.x, c.x, a.y, c.y);
                } else {
#pragma unroll
                    for (int j = 0; j < G / 2; ++j) {
                        const uint4 a = lds128(tile_s + ((2 * j) * 32 + lane) * 16);
                        const uint4 c = lds128(tile_s + ((2 * j + 1) * 32 + lane) * 16);
                        group_scores(2 * j, a.x, c.x, a.y, c.y);
                        group_scores(2 * j + 1, a.z, c.z, a.w, c.w);
                    }
                }
                if (edge) {
                    if (tok + g >= lim0) s[0] = -INFINITY;
                    if (tok + g >= lim1) s[1] = -INFINITY;
                    if (tok + g + 8 >= lim0) s[2] = -INFINITY;
                    if (tok + g + 8 >= lim1) s[3] = -INFINITY;
                }
                // a new maximum (or a scale that would not fit) anywhere in the warp: rescale what is summed
                __half2 big = __hmax2(*reinterpret_cast<const __half2*>(&vp[0][0]), *reinterpret_cast<const __half2*>(&vp[1][0]));
#pragma unroll
                for (int y = 1; y < G; ++y) {
                    big = __hmax2(big, *reinterpret_cast<const __half2*>(&vp[0][y]));
                    big = __hmax2(big, *reinterpret_cast<const __half2*>(&vp[1][y]));
                }
                float top = __low2float(big);
                if (__any_sync(0xffffffffu, s[0] > m0 || s[2] > m0 || s[1] > m1 || s[3] > m1 || top > vcap)) {
                    float n0 = fmaxf(m0, fmaxf(s[0], s[2])), n1 = fmaxf(m1, fmaxf(s[1], s[3]));
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) {
                        n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, x));
                        n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, x));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    }
                    float r0 = m0 == n0 ? 1.f : ex2(m0 - n0), r1 = m1 == n1 ? 1.f : ex2(m1 - n1);
                    m0 = n0;
                    m1 = n1;
                    l0 *= r0;
                    l1 *= r1;
#pragma unroll
                    for (int y = 0; y < G; ++y) {
                        om[y][0] *= r0;
                        om[y][1] *= r1;
                    }
                    if (top > vcap) {
                        // the largest scale becomes 2^8 .. 2^9: 7 bits of room above, 22 below to fp16's
                        // smallest normal number; never less than 2^-1, with which every finite scale fits
                        const int e = max(8 - (static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127), -1);
                        const float to = __uint_as_float(static_cast<uint32_t>(min(e, 100) + 127) << 23);
                        const float f = to / vmul;
                        vmul = to;
                        vcap = 32768.f / to;
                        r0 *= f;
                        r1 *= f;
                    }
#pragma unroll
                    for (int x = 0; x < 4 * G; ++x) {
                        o[x][0] *= r0;
                        o[x][1] *= r1;
                        o[x][2] *= r0;
                        o[x][3] *= r1;
                    }
                }
                const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
                const float p0 = ex2(s[0] - u0), p1 = ex2(s[1] - u1), p2 = ex2(s[2] - u0), p3 = ex2(s[3] - u1);
                l0 += p0 + p2;
                l1 += p1 + p3;
#pragma unroll
                for (int y = 0; y < G; ++y) {
                    const float sa = lo_f(vp[0][y]) * vmul, sb = lo_f(vp[1][y]) * vmul;
                    const float na = hi_f(vp[0][y]), nb = hi_f(vp[1][y]);
                    om[y][0] = fmaf(p0, na, fmaf(p2, nb, om[y][0]));
                    om[y][1] = fmaf(p1, na, fmaf(p3, nb, om[y][1]));
                    const __half2 ha = __floats2half2_rn(p0 * sa, p1 * sa), hb = __floats2half2_rn(p2 * sb, p3 * sb);
                    const __half2 la = __floats2half2_rn(fmaf(p0, sa, -__low2float(ha)), fmaf(p1, sa, -__high2float(ha)));
                    const __half2 lb = __floats2half2_rn(fmaf(p2, sb, -__low2float(hb)), fmaf(p3, sb, -__high2float(hb)));
                    const uint32_t b0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&ha));
                    const uint32_t b1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&hb));
                    const uint32_t e0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&la));
                    const uint32_t e1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&lb));
                    const uint4 v = lds128(tile_s + T::kV + y * 512 + lane * 16);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t a0 = w[x] & 0x000F000Fu, a1 = w[x] & 0x00F000F0u;
                        const uint32_t a2 = (w[x] >> 8) & 0x000F000Fu, a3 = (w[x] >> 8) & 0x00F000F0u;
                        mma16816(o[4 * y + x], a0, a1, a2, a3, b0, b1);
                        mma16816(o[4 * y + x], a0, a1, a2, a3, e0, e1);
                    }
                }
            }
            __syncwarp();
            if (i + S < mine) issue(i + S);
        }

        // ---- join the warps: rows relative to the CTA's maximum, summed in warp order
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, x);
            l1 += __shfl_xor_sync(0xffffffffu, l1, x);
#pragma unroll
            for (int y = 0; y < G; ++y) {
                om[y][0] += __shfl_xor_sync(0xffffffffu, om[y][0], x);
                om[y][1] += __shfl_xor_sync(0xffffffffu, om[y][1], x);
            }
        }
        if (g == 0) {
            s_max[warp * kRows + 2 * t] = m0;
            s_max[warp * kRows + 2 * t + 1] = m1;
            s_sum[warp * kRows + 2 * t] = l0;
            s_sum[warp * kRows + 2 * t + 1] = l1;
        }
        __syncthreads();  // every warp is done with its ring, too
        float top0 = -INFINITY, top1 = -INFINITY;
        for (int w = 0; w < NW; ++w) {
            top0 = fmaxf(top0, s_max[w * kRows + 2 * t]);
            top1 = fmaxf(top1, s_max[w * kRows + 2 * t + 1]);
        }
        {
            const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - top0), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - top1);
            const float k0 = f0 * (16777216.f / vmul), k1 = f1 * (16777216.f / vmul);
            float* part = reinterpret_cast<float*>(smem) + warp * kRows * C::kPitch;
#pragma unroll
            for (int x = 0; x < 4 * G; ++x) {
                const int d = 16 * x + g, y = x / 4;
                part[2 * t * C::kPitch + d] = fmaf(o[x][0], k0, om[y][0] * f0);
                part[(2 * t + 1) * C::kPitch + d] = fmaf(o[x][1], k1, om[y][1] * f1);
                part[2 * t * C::kPitch + d + 8] = fmaf(o[x][2], k0 * 0.0625f, om[y][0] * f0);
                part[(2 * t + 1) * C::kPitch + d + 8] = fmaf(o[x][3], k1 * 0.0625f, om[y][1] * f1);
            }
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == sq.tiles;
        const int64_t unit_at = seq_at + static_cast<int64_t>(unit) * sq.tiles;  // its place in the work list
        const int cta0 = static_cast<int>(unit_at / per), cta1 = static_cast<int>((unit_at + sq.tiles - 1) / per);
        float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) + kCounterBytes);
        float* my_part = parts + static_cast<int64_t>(2 * blockIdx.x + (t0 == 0 ? 1 : 0)) * C::kPart;
        auto finish = [&](int r, int d, float sum, float total, float top) {
            const int pos = (rt * kRows + r) / grp, hd = (rt * kRows + r) % grp;
            const int64_t at = static_cast<int64_t>(sq.q0 + pos) * p.heads + kvh * grp + hd;
            p.out[at * D + d] = __half_as_ushort(__float2half_rn(total > 0.f ? sum / total : 0.f));
            if (d == 0 && p.lse != nullptr)
                p.lse[at] = total > 0.f ? 0.6931471805599453f * (top + log2f(total)) : -INFINITY;
        };
        for (int x = tid; x < rows * D; x += C::kThreads) {
            const int r = x / D, d = x - r * D;
            float sum = 0.f, total = 0.f, top = -INFINITY;
            for (int w = 0; w < NW; ++w) top = fmaxf(top, s_max[w * kRows + r]);
            for (int w = 0; w < NW; ++w) {
                sum += reinterpret_cast<float*>(smem)[(w * kRows + r) * C::kPitch + d];
                const float m = s_max[w * kRows + r];
                total += m == -INFINITY ? 0.f : s_sum[w * kRows + r] * ex2(m - top);
            }
            if (whole) {
                finish(r, d, sum, total, top);
            } else {
                __stcg(my_part + 2 * kRows + x, sum);
                if (d == 0) {
                    __stcg(my_part + r, top);
                    __stcg(my_part + kRows + r, total);
                }
            }
        }
        if (!whole) {
            // ---- the last CTA of the unit to arrive adds its parts in CTA order
            unsigned* counter = static_cast<unsigned*>(p.workspace) + cta0;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const unsigned before = atomicAdd(counter, 1u);
                *s_last = before == static_cast<unsigned>(cta1 - cta0);
                if (*s_last) *counter = 0;
            }
            __syncthreads();
            if (*s_last) {
                __threadfence();
                for (int x = tid; x < rows * D; x += C::kThreads) {
                    const int r = x / D, d = x - r * D;
                    float sum = 0.f, total = 0.f, top = -INFINITY;
                    for (int c = cta0; c <= cta1; ++c)
                        top = fmaxf(top, __ldcg(parts + static_cast<int64_t>(2 * c + (c == cta0 ? 1 : 0)) * C::kPart + r));
                    for (int c = cta0; c <= cta1; ++c) {
                        const float* part = parts + static_cast<int64_t>(2 * c + (c == cta0 ? 1 : 0)) * C::kPart;
                        const float m = __ldcg(part + r);
                        const float f = m == -INFINITY ? 0.f : ex2(m - top);
                        sum = fmaf(__ldcg(part + 2 * kRows + x), f, sum);
                        total = fmaf(__ldcg(part + kRows + r), f, total);
                    }
                    finish(r, d, sum, total, top);
                }
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the ring is written by copies again
        __syncthreads();
        off += t1 - t0;
        left -= t1 - t0;
    }
}

template <int D>
cudaError_t launch_decode(const Kv4AttnParams& p, const Kv4View& v, const LaunchCtx& ctx) {
    cudaError_t e = cudaFuncSetAttribute(kv4_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Decode<D>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctx.sm_count < kMaxCtas ? ctx.sm_count : kMaxCtas), 1, 1);
    cfg.blockDim = dim3(Decode<D>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = Decode<D>::kSmem;
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_decode_kernel<D>, p, v, ctx.timeout_ns, ctx.status);
}

}  // namespace

size_t kv4_attention_workspace(int head_dim) {
    return (kCounterBytes + static_cast<size_t>(2 * kMaxCtas) * kRows * (head_dim + 2) * 4 + 15) / 16 * 16;
}

cudaError_t launch_kv4_attention(const Kv4AttnParams& p, const Kv4Cache& c, const LaunchCtx& ctx) {
    Kv4View v;
    v.pages = static_cast<uint8_t*>(c.pages);
    v.num_pages = c.num_pages;
    v.page_shift = 0;
    while ((1 << v.page_shift) < c.page_tokens) ++v.page_shift;
    v.kv_heads = c.kv_heads;
    switch (c.head_dim) {
        case 64: return launch_decode<64>(p, v, ctx);
        case 128: return launch_decode<128>(p, v, ctx);
        default: return launch_decode<256>(p, v, ctx);
    }
}

}  // namespace w4a16
