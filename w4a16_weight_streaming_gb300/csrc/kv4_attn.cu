// Attention over the 4-bit paged key/value cache for few query rows a sequence (decode and short verify
// steps): o = softmax(scale q k'^T) v', k' and v' the stored values min + code * scale.
//
// Memory-bound: every cached byte is used by the 5 or so query heads of its key/value head, times the
// queries of a verify step. The rows of one key/value head are taken 8 at a time, one column each of an
// m16n8k16 matrix instruction whose 16 rows are cached tokens (scores) or elements (output):
//   scores  S^T[16 tokens][8 rows]   = K codes [16 x D] . Q^T[D x 8]
//   output  O^T[D][8 rows]          += V codes^T [D x 16] . P[16 x 8]
// The codes go into the instruction as they are: a nibble in the low bits of an fp16 is the subnormal
// code * 2^-24, in those of a bf16 code * 2^-133, both exact, so a pair of operands costs one AND. (The
// nibbles one place up count 16 times: for keys their elements of q are divided by 16, for values they are
// other rows of the output. With them a bf16 leaves its subnormal numbers, at the same step.) The
// parameters come in around the products, in fp32, per token t and group y of 64 elements:
//   S_t  = sum_y scale_ty (sum_d q_d code_td) + min_ty (sum_d q_d)
//   O_d  = sum_t (P_t scale_ty) code_td + sum_t P_t min_ty
// P_t scale_ty 2^100 goes into the instruction as two bf16 numbers, its rounding and what that left over, 2^-18
// of itself or less: the codes' part and the minimums' part of a value cancel where the value is small, so one
// rounding would be off by 2^-9 of the group's whole range. bf16, since its exponents reach every P times every
// scale: with two fp16 numbers under a power of two of the warp's largest scale, what was below 2^-25 of that was
// lost (the values of groups with 2^-12 of another group's scale were off by 9 %).
//
// Work is a list of (sequence, 8 rows, key/value head, 16-token tile); every CTA takes an equal share of
// it, whatever the lengths, and its warps take the run's tiles in turn, each with a running maximum and
// sum of its own, so that no warp waits for another inside a run. A tile is one bulk copy into the
// warp's own ring in shared memory. Runs that end inside a row group leave their part in the workspace;
// the CTA that arrives last there adds the parts in CTA order.
//
// Measured on one GB300: one sequence of 131,072 tokens, 20 heads on 4 of 256, 40.1 us (151 MB, 3.8 TB/s, 0.56 of
// the copy bandwidth); 64 sequences of up to 8192 tokens, 40 heads on 8 of 128, 78.3 us (304 MB, 3.9 TB/s, 0.57);
// one sequence of 777 tokens 10.0 us, which is the kernel's start (4 us), a few tiles, and the adding of parts (3
// us). A tile is 371 warp instructions for D = 128 and 579 for 256; with the 16 warps that the registers leave room
// for an SM issues 2.2 of 4 a cycle, its ALU busy half of the time: the issue of dependent instructions bounds
// the long calls, not memory.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "w4a16.h"

namespace w4a16 {
namespace {

constexpr int kRows = 8;       // query rows of one work unit
// What the start and end of a unit in a CTA cost, in tiles (narrow shape, 64 sequences of 512 .. 8192 tokens
// and 8 key/value heads of 128: 93.7 us without it, the CTAs with short sequences last)
constexpr int kUnitCost = 20;

// The kernel in two shapes, the same registers and ring bytes on an SM. Wide: one CTA, for few work units
// (every CTA then has one run inside one unit, and few parts are left to add). Narrow: 3 or 4 CTAs of 4
// warps, for many units: the start and end of one CTA's run (page numbers, queries, first copies; joining
// the warps, writing) are hidden by the others' tiles.
template <int D, bool Narrow>
struct Decode {
    static constexpr int kCtas = !Narrow ? 1 : D == 256 ? 3 : 4;
    static constexpr int kWarps = Narrow ? 4 : D == 256 ? 12 : 16;
    static constexpr int kStages = D == 256 ? 3 : D == 128 ? 5 : 8;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kWhole = kWarps * (D == 256 ? 2 : D == 128 ? 3 : 4);
    static constexpr int kTile = Kv4<D>::kTileBytes;
    static constexpr int kRing = kWarps * kStages * kTile;
    static constexpr int kPitch = D + 4;  // floats between rows of a warp's part: conflict-free stores
    static constexpr int kJoin = kWarps * kRows * kPitch * 4;
    static constexpr int kData = kRing > kJoin ? kRing : kJoin;
    static constexpr int kQ = D / 64 * 1024 + 256;  // queries as operands, their sums, the rows' units
    static constexpr int kSmem = kData + kQ + kWarps * kStages * 8 + kWarps * kRows * 8 + 256;
    static constexpr int kPart = kRows * (D + 2);  // floats of one workspace part: m, l, then rows
};

// 2^100: P times scale, 2^22 at most, stays finite, and its product with a code of 2^-133 is a normal number down to
// P scale = 2^-93
constexpr float kUp = 1.2676506002282294e30f;
constexpr float kDown = 8589934592.f;  // 2^33: 1 over what a code unit times kUp is

constexpr int kMaxCtas = 640;
constexpr size_t kCounterBytes = 4096;
static_assert(kMaxCtas * 4 <= kCounterBytes, "a counter a CTA");

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// c = A . B
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma16816_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// a, b as bf16, a in the low half
__device__ __forceinline__ uint32_t pack_bf2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ float lo_bf(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
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

template <int D, bool Narrow>
__global__ void __launch_bounds__(Decode<D, Narrow>::kThreads, Decode<D, Narrow>::kCtas)
    kv4_decode_kernel(const Kv4AttnParams p, const Kv4View cache, uint64_t timeout_ns, unsigned* status) {
    using C = Decode<D, Narrow>;
    using T = Kv4<D>;
    constexpr int G = T::kGroups, NW = C::kWarps, S = C::kStages;
    constexpr int kBatch = Narrow ? 4 : 13;  // parts read at a time by the CTA that adds them
    extern __shared__ __align__(128) uint8_t smem[];
    uint4* s_q = reinterpret_cast<uint4*>(smem + C::kData);  // [G][2][32 lanes]
    uint32_t* s_qsum = reinterpret_cast<uint32_t*>(s_q + G * 2 * 32);
    float* s_unit = reinterpret_cast<float*>(s_qsum + 32);
    float* s_max = reinterpret_cast<float*>(smem + C::kData + C::kQ + NW * S * 8);  // [NW][8]
    float* s_sum = s_max + NW * kRows;
    float* s_row = s_sum + NW * kRows;  // maximum and sum of the unit's rows
    int64_t* s_plan = reinterpret_cast<int64_t*>(s_row + 2 * kRows);  // run length, offset in the first sequence
    int* s_first = reinterpret_cast<int*>(s_plan + 4);
    int* s_abort = s_first + 1;
    int* s_last = s_first + 2;
    Seq* s_seq = reinterpret_cast<Seq*>(s_first + 4);  // sequence *s_first
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * S * C::kTile;
    const uint32_t bars = smem_u32(smem + C::kData + C::kQ) + warp * S * 8;
    const int grp = p.heads / cache.kv_heads;

    if (lane == 0)
        for (int i = 0; i < S; ++i) mbar_init(bars + 8 * i, 1);
    if (tid == 0) *s_abort = 0;
    fence_barrier_init();
    griddep_launch_dependents();
    griddep_wait();

    // ---- this CTA's run of the work list
    auto chunks_of = [](int tiles, int size) { return tiles <= C::kWhole ? 1 : (tiles + size - 1) / size; };
    if (warp == 0) {
        int64_t total = 0;
        int units = 0;
        Seq seq = {};  // sequence b0 + lane; 32 or fewer are read once (each trip to memory is 0.6 us)
        auto read = [&](int b0) {
            seq = Seq{};
            if (b0 + lane < p.B) seq = seq_of(p, cache, b0 + lane);
        };
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            read(b0);
            if (seq.bad && blockIdx.x == 0) record_error(status, kErrBounds);
            int64_t c = static_cast<int64_t>(seq.units) * (seq.tiles + kUnitCost);
            const int n = min(seq.units, kMaxCtas);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
            total += c;
            units = min(kMaxCtas, units + __reduce_add_sync(0xffffffffu, n));
        }
        // Few units: each is cut into equal chunks, one a CTA, the chunk size the smallest of 32 candidates
        // with which there are CTAs enough (twice the mean is, when half the CTAs suffice for the units); a
        // tile a warp at least (one sequence of 2000 tokens, 4 heads of 256: 11.0 us, with two 12.2, with four
        // 15.0). Adding the parts takes 3 us, a tile 1.3 (256), 0.8 (128) or 0.5 (64): a unit of up to kWhole
        // tiles is left whole. Otherwise equal runs that may begin and end inside a unit.
        const int grid = static_cast<int>(gridDim.x);
        const bool chunked = 2 * units <= grid;
        int64_t per = max((total + grid - 1) / grid, static_cast<int64_t>(chunked ? NW : NW + kUnitCost));
        if (chunked) {
            const int mine = static_cast<int>(min(per + (per * lane + 30) / 31, static_cast<int64_t>(1 << 30)));
            int items = 0;
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                if (p.B > 32) read(b0);
                for (int l = 0; l < min(32, p.B - b0); ++l) {
                    const int n = __shfl_sync(0xffffffffu, seq.units, l), tiles = __shfl_sync(0xffffffffu, seq.tiles, l);
                    items += n * chunks_of(tiles, mine);
                }
            }
            const uint32_t fits = __ballot_sync(0xffffffffu, items <= grid);
            per = __shfl_sync(0xffffffffu, mine, fits ? __ffs(fits) - 1 : 31);
        }
        // where the run (its first tile, or this CTA's chunk) lies
        const int64_t w0 = chunked ? blockIdx.x : min(total, per * blockIdx.x), w1 = min(total, w0 + per);
        int64_t at = 0;
        int first = p.B;
        for (int b0 = 0; b0 < p.B && (chunked || w0 < w1); b0 += 32) {
            if (p.B > 32) read(b0);
            const int64_t c = static_cast<int64_t>(seq.units) * (chunked ? chunks_of(seq.tiles, static_cast<int>(per)) : seq.tiles + kUnitCost);
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
        if (lane == (first < p.B ? first & 31 : 0)) {
            *s_seq = seq;
            s_plan[0] = chunked ? (first < p.B ? 1 : 0) : w1 - w0;
            s_plan[1] = w0 - at;
            s_plan[2] = per;
            s_plan[3] = at;  // work list position of the first sequence
            s_first[0] = first;
            s_first[3] = chunked;
        }
    }
    __syncthreads();
    int64_t left = s_plan[0], off = s_plan[1], seq_at = s_plan[3];
    const int64_t per = s_plan[2];
    const bool chunked = s_first[3] != 0;
    uint32_t phase = 0;  // one bit per ring stage
    int copies = 0;      // that the warp has asked for
    const uint64_t policy = policy_evict_first();

    const int first = *s_first;
    for (int b = first; left > 0 && b < p.B;) {
        const Seq sq = b == first ? *s_seq : seq_of(p, cache, b);
        int unit, t0, t1, cta0, cta1;  // tiles t0 .. t1-1 of the unit, whose parts come from CTAs cta0 .. cta1
        if (chunked) {
            const int chunks = chunks_of(sq.tiles, static_cast<int>(per)), size = (sq.tiles + chunks - 1) / chunks;
            unit = static_cast<int>(off) / chunks;
            const int chunk = static_cast<int>(off) - unit * chunks;
            t0 = chunk * size;
            t1 = min(sq.tiles, t0 + size);
            cta0 = static_cast<int>(blockIdx.x) - chunk;
            cta1 = cta0 + (sq.tiles + size - 1) / size - 1;
            if (t0 >= t1) break;  // equal chunks came out one fewer
        } else {
            const int64_t each = sq.tiles + kUnitCost, cost = sq.units * each;
            if (off >= cost) {
                off -= cost;  // a sequence without rows, or done
                seq_at += cost;
                ++b;
                continue;
            }
            unit = static_cast<int>(off / each);
            const int64_t in_unit = off - unit * each, to = min(each, in_unit + left);
            t0 = static_cast<int>(max(static_cast<int64_t>(0), in_unit - kUnitCost));
            t1 = static_cast<int>(max(static_cast<int64_t>(0), to - kUnitCost));
            off += to - in_unit;
            left -= to - in_unit;
            if (t0 == t1) continue;
            const int64_t unit_at = seq_at + unit * each;  // its place in the work list
            cta0 = static_cast<int>((unit_at + kUnitCost) / per);
            cta1 = static_cast<int>((unit_at + each - 1) / per);
        }
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

        // ---- the ring: where 32 of the warp's tiles at a time lie (one a lane), one bulk copy a tile
        int64_t tile_at = -1;
        uint32_t there = 0;  // tiles in the ring whose page exists, by stage
        auto locate = [&](int i0) {
            const int tile = t0 + warp + NW * (i0 + lane);
            tile_at = -1;
            if (tile < t1e && in_bounds((tile * kKv4Tile >> cache.page_shift) < p.max_pages, status)) {
                const int tok = tile * kKv4Tile;
                const int page = p.block_table[static_cast<int64_t>(b) * p.max_pages + (tok >> cache.page_shift)];
                if (page >= 0 && page < cache.num_pages) {
                    tile_at = cache.tile_offset<D>(page, kvh, tok & ((1 << cache.page_shift) - 1));
                    if (!in_bounds(tile_at >= 0 && tile_at + C::kTile <= cache.bytes<D>(), status)) tile_at = -1;
                } else {
                    record_error(status, kErrBounds);
                }
            }
        };
        auto issue = [&](int i, int st) {
            if ((i & 31) == 0) locate(i);
            const int64_t from = __shfl_sync(0xffffffffu, tile_at, i & 31);
            there = from >= 0 ? there | (1u << st) : there & ~(1u << st);
            if (from >= 0 && lane == 0) {
                mbar_arrive_expect_tx(bars + 8 * st, C::kTile);
                if (!kDebugBounds || copies++ != p.withhold)
                    bulk_g2s(ring + st * C::kTile, cache.pages + from, C::kTile, bars + 8 * st, policy);
            }
        };
        // ---- Q^T as the B operand (row g of the unit), times a power of two that brings the row's largest
        // element to 2^8 .. 2^9: the odd pairs, whose codes count 16 times, are divided by 16 without loss.
        // Then the sums of q over each group, as two fp16 numbers: what the keys' minimums are multiplied by.
        // One warp makes them for all.
        uint4 raw[G][2];
        if (warp == 0) {
            const int pos = (rt * kRows + g) / grp, hd = (rt * kRows + g) % grp;
            const uint16_t* src = p.q + (sq.q0 + pos) * p.q_stride + static_cast<int64_t>(kvh * grp + hd) * D;
#pragma unroll
            for (int y = 0; y < G; ++y)
#pragma unroll
                for (int w = 0; w < 2; ++w)
                    raw[y][w] = g < rows && in_bounds(sq.q0 + pos < p.M, status) ? *reinterpret_cast<const uint4*>(src + y * kKv4Group + 16 * t + 8 * w)
                                         : make_uint4(0, 0, 0, 0);
        }
        // (the first copies are on their way before the queries are used)
        for (int i = 0; i < min(S, mine); ++i) issue(i, i);
        if (warp == 0) {
            float big = 0.f;
#pragma unroll
            for (int y = 0; y < G; ++y)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t v[4] = {raw[y][w].x, raw[y][w].y, raw[y][w].z, raw[y][w].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) big = fmaxf(big, fmaxf(fabsf(lo_f(v[i])), fabsf(hi_f(v[i]))));
                }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            const int e = big > 0.f && big < INFINITY ? 8 - (static_cast<int>(__float_as_uint(big) >> 23) - 127) : 0;
            const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
            float sum[G];
#pragma unroll
            for (int y = 0; y < G; ++y) {
                sum[y] = 0.f;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    uint32_t v[4] = {raw[y][w].x, raw[y][w].y, raw[y][w].z, raw[y][w].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = lo_f(v[i]) * up, c = hi_f(v[i]) * up;
                        sum[y] += a + c;
                        const float k = (i & 1) ? 0.0625f : 1.f;
                        v[i] = pack_h2(a * k, c * k);
                    }
                    s_q[(y * 2 + w) * 32 + lane] = make_uint4(v[0], v[2], v[1], v[3]);
                }
                sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 1);
                sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 2);
            }
            // columns 0 .. G-1 of the operand: the sums rounded; columns 4 ..: what is left
            uint32_t v = 0;
            if (G == 1) {
                const float r = __half2float(__float2half_rn(sum[0]));
                if ((t & 1) == 0) v = pack_h2(t == 0 ? sum[0] : sum[0] - r, 0.f);
            } else {
                const bool second = G == 4 && (t & 1);
                const float a = second ? sum[G > 2 ? 2 : 0] : sum[0], c = second ? sum[G > 2 ? 3 : 0] : sum[G > 1 ? 1 : 0];
                const float ra = a - __half2float(__float2half_rn(a)), rc = c - __half2float(__float2half_rn(c));
                if (G == 4 || (t & 1) == 0) v = t < 2 ? pack_h2(a, c) : pack_h2(ra, rc);
            }
            s_qsum[lane] = v;
            if (t == 0) s_unit[g] = p.scale * (1.4426950408889634f * 16777216.f) / up;  // scale log2(e) 2^24
        }
        __syncthreads();
        const uint32_t qsum = s_qsum[lane];
        // what takes a score of rows 2t, 2t + 1 in code units to powers of two
        const float row0 = s_unit[2 * t], row1 = s_unit[2 * t + 1];
        const uint32_t q_s = smem_u32(s_q) + lane * 16;
        float o[4 * G][4], om[G][2];
#pragma unroll
        for (int i = 0; i < 4 * G; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
        for (int y = 0; y < G; ++y) om[y][0] = om[y][1] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        for (int i = 0, st = 0; i < mine; ++i, st = st + 1 == S ? 0 : st + 1) {
            const bool have = (there >> st) & 1u;
            const uint32_t tile_s = ring + st * C::kTile;
            if (have) {
                if (!warp_suspend(bars + 8 * st, (phase >> st) & 1u, s_abort, timeout_ns, status)) {
                    // Give up: let this warp's copies in flight (of tiles i .. i + S - 1) land, bounded, before their
                    // memory is used for the parts or another CTA has it. The CTA ends with this unit.
                    for (int j = 0, k = st; j < S && i + j < mine; ++j, k = k + 1 == S ? 0 : k + 1)
                        if ((there >> k) & 1u)
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
                // scores of tokens g, g + 8 (s[0..1], s[2..3]) and rows 2t, 2t + 1
                float s[4];
                {
                    // minimums of the groups that this lane's columns of the A operand stand for
                    uint32_t ka, kb;
                    if constexpr (G == 4) {
                        ka = __byte_perm((t & 1) ? kp[0][2] : kp[0][0], (t & 1) ? kp[0][3] : kp[0][1], 0x7632);
                        kb = __byte_perm((t & 1) ? kp[1][2] : kp[1][0], (t & 1) ? kp[1][3] : kp[1][1], 0x7632);
                    } else if constexpr (G == 2) {
                        ka = __byte_perm(kp[0][0], kp[0][1], 0x7632);
                        kb = __byte_perm(kp[1][0], kp[1][1], 0x7632);
                    } else {
                        ka = kp[0][0] >> 16;
                        kb = kp[1][0] >> 16;
                    }
                    mma16816_first(s, ka, kb, 0u, 0u, qsum, 0u);
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) s[x] *= 5.9604644775390625e-8f;  // 2^-24: the unit of the codes
                auto group_scores = [&](int y, uint32_t a_w0, uint32_t b_w0, uint32_t a_w1, uint32_t b_w1) {
                    float x[4];
                    constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;
                    const uint4 q0 = lds128(q_s + (2 * y) * 512), q1 = lds128(q_s + (2 * y + 1) * 512);
                    mma16816_first(x, a_w0 & kLow, b_w0 & kLow, (a_w0 >> 8) & kLow, (b_w0 >> 8) & kLow, q0.x, q0.y);
                    mma16816(x, a_w0 & kHigh, b_w0 & kHigh, (a_w0 >> 8) & kHigh, (b_w0 >> 8) & kHigh, q0.z, q0.w);
                    mma16816(x, a_w1 & kLow, b_w1 & kLow, (a_w1 >> 8) & kLow, (b_w1 >> 8) & kLow, q1.x, q1.y);
                    mma16816(x, a_w1 & kHigh, b_w1 & kHigh, (a_w1 >> 8) & kHigh, (b_w1 >> 8) & kHigh, q1.z, q1.w);
                    const float sa = lo_f(kp[0][y]), sb = lo_f(kp[1][y]);
                    s[0] = fmaf(sa, x[0], s[0]);
                    s[1] = fmaf(sa, x[1], s[1]);
                    s[2] = fmaf(sb, x[2], s[2]);
                    s[3] = fmaf(sb, x[3], s[3]);
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
                s[0] *= row0;
                s[1] *= row1;
                s[2] *= row0;
                s[3] *= row1;
                if (edge) {
                    if (tok + g >= lim0) s[0] = -INFINITY;
                    if (tok + g >= lim1) s[1] = -INFINITY;
                    if (tok + g + 8 >= lim0) s[2] = -INFINITY;
                    if (tok + g + 8 >= lim1) s[3] = -INFINITY;
                }
                // P may grow to 2^8 before the reference moves: most tiles rescale nothing. A score above that
                // anywhere in the warp: take the new maximum, rescale the sums.
                if (__any_sync(0xffffffffu, fmaxf(s[0], s[2]) > m0 + 8.f || fmaxf(s[1], s[3]) > m1 + 8.f)) {
                    float n0 = fmaxf(m0, fmaxf(s[0], s[2])), n1 = fmaxf(m1, fmaxf(s[1], s[3]));
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) {
                        n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, x));
                        n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, x));
                    }
                    const float r0 = m0 == n0 ? 1.f : ex2(m0 - n0), r1 = m1 == n1 ? 1.f : ex2(m1 - n1);
                    m0 = n0;
                    m1 = n1;
                    l0 *= r0;
                    l1 *= r1;
#pragma unroll
                    for (int y = 0; y < G; ++y) {
                        om[y][0] *= r0;
                        om[y][1] *= r1;
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
                    const float sa = lo_f(vp[0][y]) * kUp, sb = lo_f(vp[1][y]) * kUp;
                    const float na = hi_f(vp[0][y]), nb = hi_f(vp[1][y]);
                    om[y][0] = fmaf(p0, na, fmaf(p2, nb, om[y][0]));
                    om[y][1] = fmaf(p1, na, fmaf(p3, nb, om[y][1]));
                    const uint32_t ha = pack_bf2(p0 * sa, p1 * sa), hb = pack_bf2(p2 * sb, p3 * sb);
                    const uint32_t la = pack_bf2(fmaf(p0, sa, -lo_bf(ha)), fmaf(p1, sa, -hi_bf(ha)));
                    const uint32_t lb = pack_bf2(fmaf(p2, sb, -lo_bf(hb)), fmaf(p3, sb, -hi_bf(hb)));
                    const uint32_t b0 = transpose8x8(ha), b1 = transpose8x8(hb);
                    const uint32_t e0 = transpose8x8(la), e1 = transpose8x8(lb);
                    const uint4 v = lds128(tile_s + T::kV + y * 512 + lane * 16);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        // rows g: the low codes; rows g + 8: low + 16 high (the low ones are taken off at the end)
                        const uint32_t a1 = w[x] & 0x00FF00FFu, a3 = __byte_perm(w[x], 0u, 0x4341);
                        const uint32_t a0 = w[x] & 0x000F000Fu, a2 = a3 & 0x000F000Fu;
                        mma16816_bf16(o[4 * y + x], a0, a1, a2, a3, b0, b1);
                        mma16816_bf16(o[4 * y + x], a0, a1, a2, a3, e0, e1);
                    }
                }
            }
            __syncwarp();
            if (i + S < mine) issue(i + S, st);
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
            const float k0 = f0 * kDown, k1 = f1 * kDown;
            float* part = reinterpret_cast<float*>(smem) + warp * kRows * C::kPitch;
#pragma unroll
            for (int x = 0; x < 4 * G; ++x) {
                const int d = 16 * x + g, y = x / 4;
                part[2 * t * C::kPitch + d] = fmaf(o[x][0], k0, om[y][0] * f0);
                part[(2 * t + 1) * C::kPitch + d] = fmaf(o[x][1], k1, om[y][1] * f1);
                part[2 * t * C::kPitch + d + 8] = fmaf(o[x][2] - o[x][0], k0 * 0.0625f, om[y][0] * f0);
                part[(2 * t + 1) * C::kPitch + d + 8] = fmaf(o[x][3] - o[x][1], k1 * 0.0625f, om[y][1] * f1);
            }
        }
        if (tid < kRows) {  // the CTA's maximum and sum of each row
            float top = -INFINITY, total = 0.f;
            for (int w = 0; w < NW; ++w) top = fmaxf(top, s_max[w * kRows + tid]);
            for (int w = 0; w < NW; ++w) {
                const float m = s_max[w * kRows + tid];
                total += m == -INFINITY ? 0.f : s_sum[w * kRows + tid] * ex2(m - top);
            }
            s_row[tid] = top;
            s_row[kRows + tid] = total;
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == sq.tiles;
        float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) + kCounterBytes);
        auto part_of = [&](int c) { return parts + static_cast<int64_t>(2 * c + (c == cta0 ? 1 : 0)) * C::kPart; };
        auto finish = [&](int r, int d, float4 v, float total, float top) {
            const int pos = (rt * kRows + r) / grp, hd = (rt * kRows + r) % grp;
            const int64_t at = static_cast<int64_t>(sq.q0 + pos) * p.heads + kvh * grp + hd;
            if (!in_bounds(at < static_cast<int64_t>(p.M) * p.heads && d + 4 <= D, status)) return;
            const float f = total > 0.f ? 1.f / total : 0.f;
            const __half2 h0 = __floats2half2_rn(v.x * f, v.y * f), h1 = __floats2half2_rn(v.z * f, v.w * f);
            *reinterpret_cast<uint2*>(p.out + at * D + d) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
            if (d == 0 && p.lse != nullptr)
                p.lse[at] = total > 0.f ? 0.6931471805599453f * (top + log2f(total)) : -INFINITY;
        };
        float* mine_out = part_of(blockIdx.x);
        for (int x = 4 * tid; x < rows * D; x += 4 * C::kThreads) {
            const int r = x / D, d = x - r * D;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float4 a = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem) + (w * kRows + r) * C::kPitch + d);
                v.x += a.x;
                v.y += a.y;
                v.z += a.z;
                v.w += a.w;
            }
            if (whole)
                finish(r, d, v, s_row[kRows + r], s_row[r]);
            else if (in_bounds(blockIdx.x < kMaxCtas && 2 * kRows + x + 4 <= C::kPart, status))
                __stcg(reinterpret_cast<float4*>(mine_out + 2 * kRows + x), v);
        }
        if (!whole) {
            // ---- the last CTA of the unit to arrive adds its parts in CTA order
            if (tid < 2 * kRows) __stcg(mine_out + tid, s_row[tid]);
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
                const int n = cta1 - cta0 + 1;
                float* s_f = reinterpret_cast<float*>(smem);  // [n][8]: what each part is scaled by
                for (int r = warp; r < rows; r += NW) {  // a warp per row; 64 parts' numbers in one round of loads
                    float top = -INFINITY, total = 0.f, m[2], l[2];
                    for (int c = lane; c < n; c += 64) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) m[k] = c + 32 * k < n ? __ldcg(part_of(cta0 + c + 32 * k) + r) : -INFINITY;
#pragma unroll
                        for (int k = 0; k < 2; ++k) l[k] = c + 32 * k < n ? __ldcg(part_of(cta0 + c + 32 * k) + kRows + r) : 0.f;
                        const float was = top;
                        top = fmaxf(top, fmaxf(m[0], m[1]));
                        total = was == top ? total : total * ex2(was - top);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (c + 32 * k < n) s_f[(c + 32 * k) * kRows + r] = m[k];
                            total += m[k] == -INFINITY ? 0.f : l[k] * ex2(m[k] - top);
                        }
                    }
                    const float mine_top = top;
#pragma unroll
                    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    total = mine_top == -INFINITY ? 0.f : total * ex2(mine_top - top);
#pragma unroll
                    for (int x = 16; x > 0; x >>= 1) total += __shfl_xor_sync(0xffffffffu, total, x);
                    for (int c = lane; c < n; c += 32) {
                        const float m0 = s_f[c * kRows + r];
                        s_f[c * kRows + r] = m0 == -INFINITY ? 0.f : ex2(m0 - top);
                    }
                    if (lane == 0) {
                        s_row[r] = top;
                        s_row[kRows + r] = total;
                    }
                }
                bool ready = false;
                for (int x = 4 * tid; x < rows * D || !ready; x += 4 * C::kThreads) {
                    const int r = min(x / D, rows - 1), d = x - x / D * D;
                    const bool live = x < rows * D;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int c = 0; c < n; c += kBatch) {
                        float4 a[kBatch];
#pragma unroll
                        for (int k = 0; k < kBatch; ++k)
                            a[k] = live && c + k < n
                                       ? __ldcg(reinterpret_cast<const float4*>(part_of(cta0 + c + k) + 2 * kRows + x))
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
                        if (!ready) __syncthreads();  // the factors, while the first parts are on their way
                        ready = true;
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) {
                            const float f = c + k < n ? s_f[(c + k) * kRows + r] : 0.f;
                            v.x = fmaf(a[k].x, f, v.x);
                            v.y = fmaf(a[k].y, f, v.y);
                            v.z = fmaf(a[k].z, f, v.z);
                            v.w = fmaf(a[k].w, f, v.w);
                        }
                    }
                    if (live) finish(r, d, v, s_row[kRows + r], s_row[r]);
                }
            }
        }
        // (waits run out before the warps join, so all threads read the same here; after one the ring's phases are
        // those of the copies no longer: no further unit)
        const bool over = chunked || *static_cast<volatile int*>(s_abort) != 0;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the ring is written by copies again
        __syncthreads();
        if (over) break;
    }
}

template <int D, bool Narrow>
cudaError_t launch_decode(const Kv4AttnParams& p, const Kv4View& v, const LaunchCtx& ctx) {
    using C = Decode<D, Narrow>;
    cudaError_t e = cudaFuncSetAttribute(kv4_decode_kernel<D, Narrow>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min(ctx.sm_count * C::kCtas, kMaxCtas)), 1, 1);
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_decode_kernel<D, Narrow>, p, v, ctx.timeout_ns, ctx.status);
}

// Wide where half the SMs suffice for the work units, narrow otherwise.
bool decode_is_wide(const Kv4AttnParams& p, int kv_heads, int sm_count) {
    return 2 * kv4_row_groups(p, kv_heads, kRows) * kv_heads <= sm_count;
}

template <int D>
cudaError_t launch_decode(const Kv4AttnParams& p, const Kv4View& v, bool wide, const LaunchCtx& ctx) {
    return wide ? launch_decode<D, false>(p, v, ctx) : launch_decode<D, true>(p, v, ctx);
}

// This kernel takes a pass over a sequence's tokens for every 8 query rows, the tcgen05 kernel one for every
// 128, but starts and ends slower. Fitted to 1, 16 and 64 sequences of 777 .. 16384 tokens with 1 .. 120 rows
// a key/value head, in us on 152 SMs: a start, and so much a 16-token tile of 8 rows (here) or a 64-token
// tile of 128 rows (there). Both sides, measured: 16 sequences of 4096 and 4 heads of 256, 5 rows 28.9 | 43.1,
// 10 rows 47.9 | 43.1, 20 rows 64.0 | 43.2; 8 heads of 128, 10 rows 48.7 | 57.5, 20 rows 61.0 | 57.5; 16 heads of
// 64, 20 rows 73.2 | 94.4, 40 rows 115.5 | 94.3; one sequence of 16384, heads of 256, 40 rows 31.5 | 34.4, 80 rows
// 57.3 | 41.4. The choice costs 0.3 % over the better of the two on average, 17 % at most (1000 tokens, where both
// take 20 to 35 us), where the block table is as wide as the longest sequence. The lengths are on the device and the
// table's width stands for them: with one allocated for far longer sequences several queries go to the other kernel too
// early (777 tokens under a table of 131,072, 4 heads of 256, 2 to 16 queries of 20 heads: 11.4 to 13.0 | 23.0 to
// 25.0, and the second is taken). A caller who knows the lengths names the kernel.
bool decode_is_faster(const Kv4AttnParams& p, const Kv4Cache& c, int sm_count) {
    const double start_here = c.head_dim == 256 ? 11.2 : c.head_dim == 128 ? 10.0 : 8.5;
    const double start_there = c.head_dim == 256 ? 26.3 : c.head_dim == 128 ? 19.3 : 16.1;
    const double tile_here = c.head_dim == 256 ? 0.162 : c.head_dim == 128 ? 0.087 : 0.053;
    const double tile_there = c.head_dim == 256 ? 0.73 : c.head_dim == 128 ? 0.69 : 0.74;
    const double groups = static_cast<double>(kv4_row_groups(p, c.kv_heads, kRows)), groups128 = static_cast<double>(kv4_row_groups(p, c.kv_heads, 128));
    const double tokens = static_cast<double>(p.max_pages) * c.page_tokens;
    const double here = start_here + tile_here / sm_count * c.kv_heads * groups * (tokens / kKv4Tile);
    const double there = start_there + tile_there / sm_count * c.kv_heads * groups128 * (tokens / 64);
    return here <= there;
}

}  // namespace

size_t kv4_attention_workspace(int head_dim) {
    return std::max(kv4_prompt_workspace(head_dim),
                    kCounterBytes + static_cast<size_t>(2 * kMaxCtas) * kRows * (head_dim + 2) * 4);
}

int kv4_attention_kernel(const Kv4AttnParams& p, const Kv4Cache& c, int sm_count) {
    if (p.kernel != 0) return p.kernel;
    if (decode_is_faster(p, c, sm_count)) return decode_is_wide(p, c.kv_heads, sm_count) ? W4A16_KV4_DECODE_WIDE : W4A16_KV4_DECODE;
    return kv4_prompt_pairs(p, c.kv_heads, c.head_dim) ? W4A16_KV4_PROMPT_PAIRS : W4A16_KV4_PROMPT;
}

cudaError_t launch_kv4_attention(const Kv4AttnParams& p, const Kv4Cache& c, const LaunchCtx& ctx) {
    Kv4View v;
    v.pages = static_cast<uint8_t*>(c.pages);
    v.num_pages = c.num_pages;
    v.page_shift = 0;
    while ((1 << v.page_shift) < c.page_tokens) ++v.page_shift;
    v.kv_heads = c.kv_heads;
    const int kernel = kv4_attention_kernel(p, c, ctx.sm_count);
    if (kernel == W4A16_KV4_PROMPT || kernel == W4A16_KV4_PROMPT_PAIRS)
        return launch_kv4_prompt(p, v, c.head_dim, kernel == W4A16_KV4_PROMPT_PAIRS, ctx);
    const bool wide = kernel == W4A16_KV4_DECODE_WIDE;
    switch (c.head_dim) {
        case 64: return launch_decode<64>(p, v, wide, ctx);
        case 128: return launch_decode<128>(p, v, wide, ctx);
        default: return launch_decode<256>(p, v, wide, ctx);
    }
}

}  // namespace w4a16
