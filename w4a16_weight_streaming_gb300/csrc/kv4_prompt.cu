// Attention over the 4-bit paged key/value cache for many query rows a sequence (prompt chunks, verify
// steps of several positions): o = softmax(scale q k'^T) v' on the tcgen05 tensor cores.
//
// A work unit is 128 or 256 query rows of one key/value head of one sequence (row r: query r / group, head
// r % group, so that every head that shares the keys uses one read of them) against the sequence's tokens,
// 64 at a time; for a CTA's 128 rows:
//   S[128][64]  = Q[128][D] . K'[64][D]^T      A = Q in TMEM, B = K' in shared memory
//   O[128][D]  += P[128][64] . V'[64][D]       A = P in TMEM (over S), B = V'^T in shared memory
// 256 rows are two CTAs of a cluster (cta_group::2): each keeps its rows' Q, S, P and O, dequantises half of K' (32
// tokens) and half of V' (D / 2 elements), and the first CTA issues the products of both. So a tile costs half the
// dequantisation and half the shared-memory traffic a CTA (prompt chunk of 1024 queries x 20 heads behind 8192
// tokens, 4 heads of 256: 163 us with one CTA, 141 with two).
// K', V' and P are rounded to fp16 once each (2^-11 of themselves), which the decode kernel does not do: f16 is the
// widest operand at this rate (tf32 has half of it and twice the shared memory, of which heads of 256 use all). The
// row's sum takes P before its rounding. K' and V' are fma(code, scale, min), written by dequantisation warps in
// the matrix instruction's 128-byte-swizzled layouts straight from the cache's lane order: a K word is 16 bytes of
// one token's row, a V word four pairs of tokens in rows of elements. With Q in TMEM a tile reads 64 KB of
// operands from shared memory for 1077 cycles of tensor work (D = 256), which leaves room for the dequantised
// stores; with Q in shared memory it would be 128 KB.
//
// Warps: 0-15 softmax, a quarter of a row a thread (the four warps of 32 rows meet at a barrier once a tile;
// the row's reference moves, and O is rescaled in TMEM, only when a score exceeds it by 2^8); then 8 (one CTA)
// or 4 that dequantise a 16-token quarter of the tile's keys or values each, one that fetches the cache's tiles
// by bulk copies, one that issues S and one that issues PV. K', V' and S/P are double-buffered, K' and V' of
// a pair four times. What bounds a
// tile is the circle S -> softmax -> PV -> S of its S/P buffer and the softmax warps' own chain, 1500 cycles of
// latencies, so the softmax is spread over many warps (a row in one thread: 283 us, in two 179, in four less; two
// groups of one-thread rows taking the even and the odd tiles: 186, all then with one CTA).
//
// Work is a list of (unit, tile); every CTA takes an equal run. Units that a run's end cuts leave parts
// (maximum, sum, unnormalised rows) in the workspace; the CTA that arrives last adds them, in CTA order, to
// what it still has in TMEM. (Added from memory, its own part among them: 169 us for the chunk above, 163 so.
// An SM reads parts at 45 to 60 GB/s, however many loads are under way.)
//
// Measured on one GB300: 1024 queries of 20 heads (4 of 256) behind 8192 tokens 140.9 us (183 GFLOP, 1,299 TFLOP/s,
// 0.68 of the bf16 rate); 16 sequences of 1070 .. 8005 tokens with 8 .. 16 queries each 47.0 us (73.6 MB). A tile
// of 64 tokens takes 0.95 us with 256 rows on two CTAs, of which its matrix instructions fill 0.55, 0.85 with up
// to 80 rows on one, where a tile's dequantisation (1400 cycles a warp) bounds it.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace w4a16 {
namespace {

constexpr int kRows = 128;     // query rows of a CTA
constexpr int kTok = 64;       // tokens of a tile
constexpr int kSub = kTok / kKv4Tile;
// What the start and end of a unit cost, in tiles (prompt chunk of 1024 x 20 heads behind 8192 tokens: 164.9 us
// with 6, 162.5 with 8, 163.3 with 10)
constexpr int kUnitCost = 8;
// Fewest tiles of a run: less makes more parts than it saves (24 queries of 20 heads behind 4096 tokens, 4 heads of
// 256: 32.2 us with 4, 34.8 with 8, 37.3 with 12; behind 16384 53.4, 50.0, 50.9)
constexpr int kMinRun = 6;
constexpr int kDequant = 16;   // softmax warps; the dequantising ones follow, then the fetching one and the two issuers
constexpr int kJoinInPlace = 8;  // most parts of a unit that its last CTA adds to its own in TMEM
constexpr int kNotes = 16;     // tiles whose page validity is kept
// A weight of the row's reference is 2^kLift, so that with scores up to 2^8 above it fp16 is used to 2^15, and to
// 2^-32 of the reference below (a long context beside one token that has nearly all of the weight).
constexpr float kLift = 7.f;

template <int D, bool Pair>
struct Prompt {
    static constexpr int kCtas = Pair ? 2 : 1;            // of a cluster, on one unit
    static constexpr int kUnitRows = kRows * kCtas;
    static constexpr int kTokCta = kTok / kCtas;          // tokens of K' in a CTA (of V' it has D / kCtas elements)
    // dequantising warps, half of them for keys (prompt chunk below, pair: 149 us with 8, 141 with 4)
    static constexpr int kDeq = Pair ? 4 : 8;
    static constexpr int kProducer = kDequant + kDeq, kIssueS = kProducer + 1, kThreads = (kProducer + 3) * 32;
    static constexpr int kRaw = kSub * Kv4<D>::kTileBytes;
    static constexpr int kRawStages = D == 256 ? 3 : 4;
    static constexpr int kBuf = kTok * D * 2 / kCtas;  // one K' or V' buffer
    // K' (and V') buffers. A pair's take half of the memory, and four hide what handing one to the other CTA takes
    // (prompt chunk below: 156 us with two)
    static constexpr int kBufs = Pair ? 4 : 2;
    static constexpr int kOffV = kBufs * kBuf;
    // (where the tiles are, a unit's parts are added: four slots or more of 16 elements of a part for every
    // softmax thread, or what up to kKv4MaxPromptCtas parts are scaled by, under the raw tiles)
    static constexpr int kOffRaw = 4 * 64 * kDequant * 32;
    static_assert(2 * kBufs * kBuf <= kOffRaw && kKv4MaxPromptCtas * kRows * 4 <= kOffRaw, "");
    static constexpr int kOffBars = kOffRaw + kRawStages * kRaw;
    static constexpr int kBars = 2 * kRawStages + 2 * 3 + 3 + (Pair ? 4 : 2) * kBufs;
    static constexpr int kOffMisc = kOffBars + kBars * 8;
    static constexpr int kJoin = (kJoinInPlace + 1) * kRows * 4;
    static constexpr int kSmem = kOffMisc + 256 + kJoin + 1024;  // + alignment
    static constexpr uint32_t kColS = D, kColQ = D + 2 * kTok;
    static constexpr uint32_t kCols = D == 64 ? 256 : 512;
    static constexpr int kPart = kRows * (D + 2);  // floats of one workspace part: m, l, then [D / 4][128] float4
};

// One lane of a converged warp, in a form from which the compiler sees that a single thread runs what it
// guards: a tcgen05.mma of 64 columns is then issued every 32-42 cycles (its execution time), against 64-80
// under a comparison of the lane number.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b32 r;\n\telect.sync r|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Consecutive TMEM columns of a warp's 32 lanes
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// Whether the predicate holds for any of the 128 threads that meet at named barrier `id`.
__device__ __forceinline__ bool any_of_128(int id, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred pi, po;\n\tsetp.ne.u32 pi, %1, 0;\n\tbarrier.red.or.pred po, %2, 128, pi;\n\tselp.u32 %0, 1, 0, po;\n\t}"
        : "=r"(r)
        : "r"(pred ? 1u : 0u), "r"(id)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// pairs of fp32 numbers
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// Four 8 x 8 matrices of fp16 from a warp's fragments (lane 4 g + t: row g, columns 2t, 2t + 1) to rows of
// 16 bytes; lane l gives the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
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

// The codes of a word as fp16 pairs, exact: out[i] = (nibble i, nibble i + 4).
__device__ __forceinline__ void codes(uint32_t w, uint32_t (&out)[4]) {
    constexpr uint32_t kMagic = 0x64006400u, kNeg1024 = 0xE400E400u, kSixteenth = 0x2C002C00u, kNeg64 = 0xD400D400u;
    const uint32_t hi = w >> 8;
    out[0] = hadd2(and_or(w, 0x000F000Fu, kMagic), kNeg1024);
    out[1] = hfma2(and_or(w, 0x00F000F0u, kMagic), kSixteenth, kNeg64);
    out[2] = hadd2(and_or(hi, 0x000F000Fu, kMagic), kNeg1024);
    out[3] = hfma2(and_or(hi, 0x00F000F0u, kMagic), kSixteenth, kNeg64);
}

__device__ __forceinline__ void cp_async16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ uint32_t ld_acquire(const unsigned* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

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

template <int kUnitRows>
struct PromptSeqOf {
    int q0, q_len, n, grp, row_tiles;
    bool bad;  // (24 bytes)
    // tokens that query row r (within the sequence) sees
    __device__ __forceinline__ int seen(int r, int causal) const {
        return causal ? max(0, n - (q_len - 1 - r / grp)) : n;
    }
    // tiles of a row tile (its last row sees most); at least one, so that empty rows are written
    __device__ __forceinline__ int tiles(int rt, int causal) const {
        const int last = min(q_len * grp, (rt + 1) * kUnitRows) - 1;
        const int most = seen(last, causal);
        return most > 0 ? (most - 1) / kTok + 1 : 1;  // (no sum: a length may be next to 2^31)
    }
    // The work list's unit is 1 / grp of a token: row tile rt takes a fixed cost, then no less than its
    // tokens, grows by kUnitRows from one row tile to the next (causal), and so has a sum in closed form. Its
    // tile t begins at fixed() + t * grp * kTok.
    __device__ __forceinline__ int64_t fixed() const { return static_cast<int64_t>(grp) * kTok * kUnitCost; }
    __device__ __forceinline__ int64_t flat(int causal) const {
        return fixed() + static_cast<int64_t>(grp) * (causal ? max(n - q_len, 0) + 1 : max(n, 1));
    }
    __device__ __forceinline__ int64_t length(int rt, int causal) const {
        return flat(causal) + (causal ? static_cast<int64_t>(rt + 1) * kUnitRows : 0);
    }
    __device__ __forceinline__ int64_t before(int rt, int causal) const {  // of row tiles 0 .. rt-1 of one head
        return rt * flat(causal) + (causal ? static_cast<int64_t>(rt) * (rt + 1) / 2 * kUnitRows : 0);
    }
};

template <int kUnitRows>
__device__ __forceinline__ PromptSeqOf<kUnitRows> prompt_seq(const Kv4AttnParams& p, const Kv4View& c, int b) {
    PromptSeqOf<kUnitRows> s;
    const int q0 = p.q_start[b], q1 = p.q_start[b + 1], n = p.kv_len[b];
    s.q0 = min(max(q0, 0), p.M);
    const int end = min(max(q1, s.q0), p.M);
    s.q_len = end - s.q0;
    s.n = min(max(n, 0), p.max_pages << c.page_shift);
    s.bad = s.q0 != q0 || end != q1 || s.n != n;
    s.grp = p.heads / c.kv_heads;
    s.row_tiles = (s.q_len * s.grp + kUnitRows - 1) / kUnitRows;
    return s;
}

// The same for the two CTAs of a cluster: one product of 256 rows, A and D in the TMEM of both (128 rows each), B
// half in each one's shared memory; issued by the cluster's first CTA.
__device__ __forceinline__ void umma_pair_f16_ts(uint32_t d_taddr, uint32_t a_taddr, uint64_t b_desc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_taddr),
        "r"(a_taddr), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void umma_pair_commit(uint32_t bar) {  // arrives at the barrier of both
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"(static_cast<uint16_t>(3))
                 : "memory");
}
__device__ __forceinline__ void tmem_pair_alloc(uint32_t slot_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot_smem), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_pair_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Arrive at the first CTA's barrier after this thread's tcgen05 instructions (tcgen05.fence::before_thread_sync here,
// after_thread_sync there order them; an arrival between the two need not release anything else).
__device__ __forceinline__ void mbar_arrive_first(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(map_peer(bar, 0)) : "memory");
}
template <int D, bool Pair>
__global__ void __launch_bounds__(Prompt<D, Pair>::kThreads, 1)
    kv4_prompt_kernel(const Kv4AttnParams p, const Kv4View cache, uint64_t timeout_ns, unsigned* status) {
    using C = Prompt<D, Pair>;
    using T = Kv4<D>;
    using PromptSeq = PromptSeqOf<C::kUnitRows>;
    auto seq_of = [](const Kv4AttnParams& p, const Kv4View& c, int b) { return prompt_seq<C::kUnitRows>(p, c, b); };
    constexpr int G = T::kGroups, R = C::kRawStages, kProducer = C::kProducer, kIssueS = C::kIssueS, kThreads = C::kThreads;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
    int* s_misc = reinterpret_cast<int*>(smem + C::kOffMisc);
    int* s_abort = s_misc;
    int* s_last = s_misc + 1;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_misc + 2);
    int* s_first = s_misc + 3;
    int* s_joined = s_misc + 30;
    int64_t* s_plan = reinterpret_cast<int64_t*>(s_misc + 4);      // run begin, end, length; first sequence's place
    uint32_t* s_valid = reinterpret_cast<uint32_t*>(s_misc + 12);  // [kNotes]: valid tokens of each quarter, a byte each
    float* s_part = reinterpret_cast<float*>(smem + C::kOffMisc + 256);  // [4][128]: what the quarters of a row exchange
    float* s_join = s_part;  // [kJoinInPlace + 1][128]: what the threads that add a unit's parts exchange
    PromptSeq* s_seq = reinterpret_cast<PromptSeq*>(s_misc + 48);  // the sequence that the run begins in
    volatile int* s_left = s_misc + 32;  // [16]: softmax warps whose wait ran out
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t bars = base + C::kOffBars;
    auto raw_full = [&](int s) { return bars + 8 * s; };
    auto raw_empty = [&](int s) { return bars + 8 * (R + s); };
    auto s_full = [&](int s) { return bars + 8 * (2 * R + s); };       // S in TMEM
    auto p_full = [&](int s) { return bars + 8 * (2 * R + 2 + s); };
    auto pv_done = [&](int s) { return bars + 8 * (2 * R + 4 + s); };  // O updated, S/P free
    const uint32_t q_full = bars + 8 * (2 * R + 6);
    auto drained = [&](int i) { return bars + 8 * (2 * R + 7 + i); };  // the issuers' instructions, after a wait ran out
    constexpr int KB = C::kBufs;
    auto k_full = [&](int s) { return bars + 8 * (2 * R + 9 + s); };
    auto v_full = [&](int s) { return bars + 8 * (2 * R + 9 + KB + s); };
    // K' and V' are free again: with two buffers at the barriers of S and O
    auto k_free = [&](int s) { return KB == 2 ? s_full(s) : bars + 8 * (2 * R + 9 + 2 * KB + s); };
    auto v_free = [&](int s) { return KB == 2 ? pv_done(s) : bars + 8 * (2 * R + 9 + 3 * KB + s); };
    // A pair's barriers for what its products read are the first CTA's. Of Q and P every warp arrives there itself. K'
    // and V' are shared memory, which takes a release at the cluster's scope to be handed to another CTA's thread: that
    // waits 900 cycles (with every warp's arrival a chunk took 186 us), so the second CTA's warps arrive at its own
    // barrier, and its issuers, which have no products to issue, pass that on while the next tile is dequantised.
    const uint32_t rank = Pair ? cluster_ctarank() : 0u;
    const int team = static_cast<int>(blockIdx.x) / C::kCtas, teams = static_cast<int>(gridDim.x) / C::kCtas;
    auto arrive = [&](uint32_t bar) {
        if constexpr (Pair) mbar_arrive_first(bar);
        else mbar_arrive(bar);
    };
    auto wait = [&](uint32_t bar, uint32_t parity) { return warp_suspend(bar, parity, s_abort, timeout_ns, status); };
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
        if constexpr (Pair) return warp_poll_cluster(bar, parity, s_abort, timeout_ns, status);
        else return warp_suspend(bar, parity, s_abort, timeout_ns, status);
    };
    auto multiply = [&](uint32_t d, uint32_t a, uint64_t desc, uint32_t idesc, bool more) {
        if constexpr (Pair) umma_pair_f16_ts(d, a, desc, idesc, more);
        else umma_f16_ts(d, a, desc, idesc, more);
    };
    // (the second CTA's issuers) the buffer is complete here: say so to the first CTA
    auto pass_on = [&](uint32_t bar, uint32_t parity) {
        if (!wait(bar, parity)) return false;
        if (lane == 0) mbar_arrive_remote(bar, 0);
        __syncwarp();
        return true;
    };
    auto commit = [&](uint32_t bar) {
        if constexpr (Pair) umma_pair_commit(bar);
        else umma_commit(bar);
    };

    if (warp == kProducer) {
        if (lane == 0) {
            for (int i = 0; i < R; ++i) {
                mbar_init(raw_full(i), 1);
                mbar_init(raw_empty(i), C::kDeq);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(s_full(i), 1);
                mbar_init(p_full(i), 16 * C::kCtas);
                mbar_init(pv_done(i), 1);
            }
            for (int i = 0; i < KB; ++i) {
                mbar_init(k_full(i), C::kDeq / 2 + (Pair && rank == 0 ? 1 : 0));
                mbar_init(v_full(i), C::kDeq / 2 + (Pair && rank == 0 ? 1 : 0));
                if constexpr (KB > 2) {
                    mbar_init(k_free(i), 1);
                    mbar_init(v_free(i), 1);
                }
            }
            mbar_init(q_full, 16 * C::kCtas);
            mbar_init(drained(0), 1);
            mbar_init(drained(1), 1);
            *s_abort = 0;
            fence_barrier_init();
        }
        __syncwarp();
        if constexpr (Pair) {
            tmem_pair_alloc(smem_u32(s_tmem), C::kCols);
        } else {
            tmem_alloc(smem_u32(s_tmem), C::kCols);
            tmem_relinquish();
        }
    }
    griddep_wait();

    // ---- this CTA's run of the work list
    if (warp == 0) {
        int64_t total = 0, cost = 0;  // cost: of sequence b0 + lane, kept for the search where there are no more than 32
        PromptSeq seq = {};
        auto read = [&](int b0) {
            cost = 0;
            if (b0 + lane < p.B) {
                seq = seq_of(p, cache, b0 + lane);
                cost = seq.before(seq.row_tiles, p.causal) * cache.kv_heads;
            }
        };
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            read(b0);
            if (b0 + lane < p.B && seq.bad && blockIdx.x == 0) record_error(status, kErrBounds);
            int64_t c = cost;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
            total += c;
        }
        const int64_t per = max((total + teams - 1) / teams,
                                static_cast<int64_t>(kMinRun + kUnitCost) * kTok * (p.heads / cache.kv_heads));
        const int64_t w0 = min(total, per * team), w1 = min(total, w0 + per);
        int64_t at = 0;
        int first = p.B;
        for (int b0 = 0; b0 < p.B && w0 < w1; b0 += 32) {
            if (p.B > 32) read(b0);
            int64_t upto = cost;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, at + upto > w0);
            if (hit != 0) {
                const int l = __ffs(hit) - 1;
                first = b0 + l;
                at += __shfl_sync(0xffffffffu, upto - cost, l);
                break;
            }
            at += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (lane == (first < p.B ? first & 31 : 0)) {
            int kvh = 0, rt = 0;
            if (first < p.B) {  // the unit that the run begins in
                const PromptSeq& s = seq;
                const int64_t head = s.before(s.row_tiles, p.causal);
                kvh = static_cast<int>((w0 - at) / head);
                at += kvh * head;
                int hi = s.row_tiles - 1;
                while (rt < hi) {
                    const int mid = (rt + hi + 1) / 2;
                    if (at + s.before(mid, p.causal) <= w0) rt = mid;
                    else hi = mid - 1;
                }
                at += s.before(rt, p.causal);
            }
            s_plan[0] = w0;
            s_plan[1] = w1;
            s_plan[2] = per;
            s_plan[3] = at;
            s_first[0] = first;
            s_first[8 + kNotes + 1] = kvh;
            s_first[8 + kNotes + 2] = rt;
            *s_seq = seq;
        }
    }
    tc_fence_before();
    __syncwarp();
    if constexpr (Pair) cluster_sync_all();  // (the other's barriers are there too)
    else __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();  // (after the allocation: the next grid's cannot come before it)
    const uint32_t tmem = *s_tmem;
    const int64_t w0 = s_plan[0], w1 = s_plan[1], per = s_plan[2];
    int64_t at = s_plan[3];  // work list position of the current unit
    int b = s_first[0], kvh = s_first[8 + kNotes + 1], rt = s_first[8 + kNotes + 2];
    uint32_t done = 0;       // tiles of earlier segments
    uint32_t segment = 0;
    uint32_t issued = 0;     // tiles that the fetching warp has asked for
    PromptSeq sq = {};
    if (b < p.B) sq = *s_seq;

    // CTA c's part of the unit that begins in CTA cta0 (of a pair, every second CTA has the same rows)
    auto part_of = [&](int cta0, int c) {
        return reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) + 4096) + static_cast<int64_t>(2 * c + (c == cta0 ? 1 : 0)) * C::kPart;
    };

    while (at < w1 && b < p.B) {
        if (rt >= sq.row_tiles) {
            rt = 0;
            if (++kvh >= cache.kv_heads || sq.row_tiles == 0) {
                kvh = 0;
                if (++b < p.B) sq = seq_of(p, cache, b);
            }
            continue;
        }
        // tiles of the unit whose places lie in the run
        const int tiles = sq.tiles(rt, p.causal), row0 = rt * C::kUnitRows + static_cast<int>(rank) * kRows;
        const int64_t first_at = at + sq.fixed(), each = static_cast<int64_t>(sq.grp) * kTok;
        const int t0 = static_cast<int>(min(static_cast<int64_t>(tiles), (max(w0 - first_at, static_cast<int64_t>(0)) + each - 1) / each));
        const int t1 = static_cast<int>(min(static_cast<int64_t>(tiles), (max(w1 - first_at, static_cast<int64_t>(0)) + each - 1) / each));
        at += sq.length(rt, p.causal);
        ++rt;
        if (t0 >= t1) continue;
        const int nt = t1 - t0;
        const int cta0 = static_cast<int>(first_at / per) * C::kCtas + static_cast<int>(rank);
        const int cta1 = static_cast<int>((first_at + (tiles - 1) * each) / per) * C::kCtas + static_cast<int>(rank);
        const int parts = (cta1 - cta0) / C::kCtas + 1;
        const int rows = max(0, min(kRows, sq.q_len * sq.grp - row0));  // (none: the second half of a pair's unit)
        const bool whole = t0 == 0 && t1 == tiles;

        if (warp < kDequant) {
            // ================= softmax: quarter `part` of row `r` of the unit
            const int quad = warp & 3, part = warp >> 2, r = quad * 32 + lane;
            const uint32_t lanes = tmem + (static_cast<uint32_t>(quad) << 21);  // this warp's 32 lanes
            const bool idle = quad * 32 >= rows;
            const int in_seq = row0 + min(r, rows - 1), pos = in_seq / sq.grp, hd = in_seq - pos * sq.grp;
            const int64_t q_row = sq.q0 + pos;
            const int head = kvh * sq.grp + hd;
            {
                const uint16_t* src = p.q + q_row * p.q_stride + static_cast<int64_t>(head) * D + part * (D / 4);
                const uint32_t sign = p.scale < 0.f ? 0x80008000u : 0u;
                uint4 x[D / 32];
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    x[c] = make_uint4(0, 0, 0, 0);
                    if (r < rows && in_bounds(q_row < p.M, status)) x[c] = *reinterpret_cast<const uint4*>(src + c * 8);
                }
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const uint32_t v[8] = {x[2 * c].x ^ sign,     x[2 * c].y ^ sign,     x[2 * c].z ^ sign,     x[2 * c].w ^ sign,
                                           x[2 * c + 1].x ^ sign, x[2 * c + 1].y ^ sign, x[2 * c + 1].z ^ sign, x[2 * c + 1].w ^ sign};
                    tmem_st8(lanes + C::kColQ + part * (D / 8) + 8 * c, v);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(q_full);
            }
            const float c1 = fmaxf(fabsf(p.scale) * 1.4426950408889634f, 1e-30f);
            const int lim = sq.seen(in_seq, p.causal);
            const int lim_min = sq.seen(row0 + min(quad * 32, rows - 1), p.causal);
            float m = -INFINITY, l = 0.f;  // the row's reference, and this quarter's sum
            bool ok = true;
            for (int i = 0; i < nt; ++i) {
                const uint32_t it = done + i, buf = it & 1, ph = (it >> 1) & 1;
                // (a warp whose wait ran out goes on to the barrier, where the four agree to leave)
                ok = ok && wait(s_full(buf), ph);
                if (idle && !ok) break;
                if (!idle) {
                    tc_fence_after();
                    const uint32_t from = lanes + C::kColS + buf * kTok;
                    uint32_t s[16];
                    tmem_ld16(from + part * 16, s);
                    tmem_wait_ld();
                    const int tok = (t0 + i) * kTok + part * 16;
                    const int there = static_cast<int>((s_valid[it % kNotes] >> (8 * part)) & 255u);
                    if (tok > lim_min - 16 || there != 16) {
                        const int most = min(there, lim - tok);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (j >= most) s[j] = 0xFF800000u;  // -inf
                    }
                    float mx = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1])), my = fmaxf(__uint_as_float(s[2]), __uint_as_float(s[3]));
#pragma unroll
                    for (int j = 4; j < 16; j += 4) {
                        mx = max3(mx, __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
                        my = max3(my, __uint_as_float(s[j + 2]), __uint_as_float(s[j + 3]));
                    }
                    mx = fmaxf(mx, my) * c1;
                    // all quarters have read S from here on: P may take its place
                    if (any_of_128(1 + quad, mx > m + 8.f || !ok)) {
                        s_part[part * kRows + r] = mx;
                        if (lane == 0) s_left[warp] = !ok;
                        named_sync(1 + quad, 128);
                        const bool leave = s_left[quad] || s_left[quad + 4] || s_left[quad + 8] || s_left[quad + 12];
                        const float now = max3(max3(m, s_part[r], s_part[kRows + r]), s_part[2 * kRows + r], s_part[3 * kRows + r]);
                        const float f = m == now ? 1.f : ex2(m - now);
                        m = now;
                        l *= f;
                        if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
                            const uint32_t before = it - 1;
                            ok = ok && wait(pv_done(before & 1), (before >> 1) & 1);
                            tc_fence_after();
#pragma unroll 1
                            for (int c = part * (D / 4); c < (part + 1) * (D / 4); c += 16) {
                                uint32_t v[16];
                                tmem_ld16(lanes + c, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * f);
                                tmem_st<16>(lanes + c, v);
                            }
                            tmem_wait_st();
                        }
                        named_sync(1 + quad, 128);  // s_part may be written again
                        if (leave) break;
                    }
                    const float sub = m == -INFINITY ? 0.f : m - kLift;
                    uint32_t pk[8];
                    uint64_t sum = 0;  // two fp32 sums
                    const uint64_t c2 = pair(c1, c1), sub2 = pair(-sub, -sub);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float a, e;
                        unpair(fma2(pair(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), c2, sub2), a, e);
                        a = ex2(a);
                        e = ex2(e);
                        sum = add2(sum, pair(a, e));
                        const __half2 x = __floats2half2_rn(a, e);
                        pk[j] = *reinterpret_cast<const uint32_t*>(&x);
                    }
                    float a, e;
                    unpair(sum, a, e);
                    l += a + e;
                    tmem_st8(from + part * 8, pk);
                    tmem_wait_st();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) arrive(p_full(buf));
            }
            // ---- the unit's rows, or this CTA's part of them: a quarter of the elements each. The last CTA adds
            // the others' parts to its own in TMEM, which is not written where they are all there by now.
            const int n = parts, own = (static_cast<int>(blockIdx.x) - cta0) / C::kCtas;
            bool join = false;
            if (!whole) {
                if (tid == 0) {
                    unsigned* counter = static_cast<unsigned*>(p.workspace) + cta0;
                    const bool there = n <= kJoinInPlace && ld_acquire(counter) == static_cast<unsigned>(n - 1);
                    if (there) *counter = 0;
                    *s_joined = there;
                    *s_last = 0;
                }
                named_sync(5, kDequant * 32);
                join = *s_joined;
            }
            if (ok) {
                const uint32_t end = done + nt - 1;
                ok = wait(pv_done(end & 1), (end >> 1) & 1);
            }
            if (!idle) {
                s_part[part * kRows + r] = l;
                named_sync(1 + quad, 128);
                l = (s_part[r] + s_part[kRows + r]) + (s_part[2 * kRows + r] + s_part[3 * kRows + r]);
                ok = !any_of_128(1 + quad, !ok);  // (the four leave together)
            }
            if (ok && !idle && !join) {
                tc_fence_after();
                const float inv = l > 0.f ? 1.f / l : 0.f;
                float* dst = reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) + 4096) +
                             static_cast<int64_t>(2 * blockIdx.x + (t0 == 0 ? 1 : 0)) * C::kPart;
                uint16_t* out = p.out + (q_row * p.heads + head) * D;
#pragma unroll 1
                for (int c = part * (D / 4); c < (part + 1) * (D / 4); c += 16) {
                    uint32_t v[16];
                    tmem_ld16(lanes + c, v);
                    tmem_wait_ld();
                    if (r >= rows || !in_bounds(q_row < p.M && blockIdx.x < kKv4MaxPromptCtas, status)) continue;
                    if (whole) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t h[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const __half2 x = __floats2half2_rn(l > 0.f ? __uint_as_float(v[8 * j + 2 * k]) * inv : 0.f,
                                                                    l > 0.f ? __uint_as_float(v[8 * j + 2 * k + 1]) * inv : 0.f);
                                h[k] = *reinterpret_cast<const uint32_t*>(&x);
                            }
                            *reinterpret_cast<uint4*>(out + c + 8 * j) = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            __stcg(reinterpret_cast<uint4*>(dst + 2 * kRows) + (c / 4 + j) * kRows + r,
                                   make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
                    }
                }
                if (r < rows && part == 0) {
                    if (!whole) {
                        __stcg(dst + r, m);
                        __stcg(dst + kRows + r, l);
                    } else if (p.lse != nullptr) {
                        p.lse[q_row * p.heads + head] = l > 0.f ? 0.6931471805599453f * (m - kLift + log2f(l)) : -INFINITY;
                    }
                }
                tc_fence_before();
            }
            if (!whole && !join) {  // this CTA's part is written: whether it was the last
                __threadfence();
                named_sync(5, kDequant * 32);
                if (tid == 0) {
                    unsigned* counter = static_cast<unsigned*>(p.workspace) + cta0;
                    *s_last = atomicAdd(counter, 1u) == static_cast<unsigned>(n - 1);
                    if (*s_last) *counter = 0;
                }
                named_sync(5, kDequant * 32);
                join = *s_last && n <= kJoinInPlace;
            }
            if (join && ok && !idle) {
                __threadfence();
                // The others' elements come through four slots of shared memory (K' and V' are not in use), 16
                // elements of one part a thread in each, every thread its own; parts in CTA order.
                constexpr int kChunks = D / 64, kSlot = 64 * kDequant * 32;
                const int rr = min(r, rows - 1);
                const uint32_t slots = base + tid * 16;
                const float4* rest = reinterpret_cast<const float4*>(part_of(cta0, cta0) + 2 * kRows) + part * (D / 16) * kRows + rr;
                int to_come = r < rows ? kChunks * (n - 1) : 0, next = own == 0, at_chunk = 0;
                uint32_t to_slot = slots;
                auto fetch = [&]() {  // part `next` of the next chunk
                    if (to_come > 0) {
                        // (the parts of the unit's other CTAs: every second one from the first's neighbour on)
                        const float4* from = rest + (next == 0 ? 0 : (2 * C::kCtas * next - 1) * (C::kPart / 4)) + at_chunk;
#pragma unroll
                        for (int k = 0; k < 4; ++k) cp_async16(to_slot + k * (kSlot / 4), from + k * kRows);
                        --to_come;
                        to_slot = to_slot == slots + 3 * kSlot ? slots : to_slot + kSlot;
                        next += next + 1 == own ? 2 : 1;
                        if (next >= n) {
                            next = own == 0;
                            at_chunk += 4 * kRows;
                        }
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                };
                for (int j = 0; j < 4; ++j) fetch();
                if (part == 0) {  // the row's factors and sum
                    float mm[kJoinInPlace], ll[kJoinInPlace], top = -INFINITY, total = 0.f;
#pragma unroll
                    for (int c = 0; c < kJoinInPlace; ++c) {
                        const float* from = part_of(cta0, cta0 + C::kCtas * min(c, n - 1)) + rr;
                        mm[c] = c == own ? m : c < n ? __ldcg(from) : -INFINITY;
                        ll[c] = c == own ? l : c < n ? __ldcg(from + kRows) : 0.f;
                        top = fmaxf(top, mm[c]);
                    }
#pragma unroll
                    for (int c = 0; c < kJoinInPlace; ++c) {
                        const float f = mm[c] == -INFINITY ? 0.f : ex2(mm[c] - top);
                        total = fmaf(ll[c], f, total);
                        if (c < n) s_join[c * kRows + r] = f;
                    }
                    s_join[kJoinInPlace * kRows + r] = total > 0.f ? 1.f / total : 0.f;
                    if (r < rows && p.lse != nullptr)
                        p.lse[q_row * p.heads + head] = total > 0.f ? 0.6931471805599453f * (top - kLift + log2f(total)) : -INFINITY;
                }
                named_sync(1 + quad, 128);
                tc_fence_after();
                const float inv = s_join[kJoinInPlace * kRows + r];
                uint16_t* out = p.out + (q_row * p.heads + head) * D + part * (D / 4);
                uint32_t slot = slots;
#pragma unroll 1
                for (int chunk = 0; chunk < kChunks; ++chunk) {
                    uint32_t v[16];
                    float sum[16];
                    tmem_ld16(lanes + part * (D / 4) + 16 * chunk, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) sum[e] = 0.f;
                    for (int c = 0; c < n; ++c) {
                        const float f = s_join[c * kRows + r];
                        if (c != own) {
                            asm volatile("cp.async.wait_group 3;" ::: "memory");
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint4 a = lds128(slot + k * (kSlot / 4));
                                if (f != 0.f) {  // (a part that saw nothing may hold anything)
                                    sum[4 * k] = fmaf(__uint_as_float(a.x), f, sum[4 * k]);
                                    sum[4 * k + 1] = fmaf(__uint_as_float(a.y), f, sum[4 * k + 1]);
                                    sum[4 * k + 2] = fmaf(__uint_as_float(a.z), f, sum[4 * k + 2]);
                                    sum[4 * k + 3] = fmaf(__uint_as_float(a.w), f, sum[4 * k + 3]);
                                }
                            }
                            slot = slot == slots + 3 * kSlot ? slots : slot + kSlot;
                            fetch();
                        } else if (f != 0.f) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) sum[e] = fmaf(__uint_as_float(v[e]), f, sum[e]);
                        }
                    }
                    if (r < rows && in_bounds(q_row < p.M, status)) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t h[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __half2 x = __floats2half2_rn(sum[8 * k + 2 * e] * inv, sum[8 * k + 2 * e + 1] * inv);
                                h[e] = *reinterpret_cast<const uint32_t*>(&x);
                            }
                            *reinterpret_cast<uint4*>(out + 16 * chunk + 8 * k) = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                    }
                }
                tc_fence_before();
            }
        } else if (warp < kProducer) {
            // ================= dequantise: keys or values of a quarter of the tokens (of values, where a CTA has half
            // of the elements, of two quarters)
            const int dw = warp - kDequant;
            const bool is_k = dw < C::kDeq / 2;
            constexpr int kValues = C::kCtas;
            const int sub0 = is_k ? 2 * static_cast<int>(rank) + dw : (dw - C::kDeq / 2) * kValues;
            const int g = lane >> 2, t = lane & 3;
            const uint32_t to_k0 = base + (dw * 16 + g) * 128;  // the row of token g
            // the 16 bytes that this lane addresses of the four 8 x 8 matrices of a V word: matrix lane / 8 (rows
            // 8 (m & 1) on, tokens 8 (m / 2) on), row lane % 8
            const uint32_t to_v0 = base + C::kOffV + (((lane >> 3) & 1) * 8 + (lane & 7)) * 128 +
                                   (((2 * sub0 + (lane >> 4)) ^ (lane & 7)) << 4);
            const uint32_t to_v1 = to_v0 ^ 32u;  // of the quarter after an even one
            for (int i = 0; i < nt; ++i) {
                const uint32_t it = done + i, st = it % R, buf = it % KB, use = it / KB;
                const uint32_t to_k = to_k0 + buf * C::kBuf;
                if (!wait(raw_full(st), (it / R) & 1)) break;
                const uint32_t note = s_valid[it % kNotes];
                if (!wait(is_k ? k_free(buf) : v_free(buf), (use & 1) ^ 1)) break;
                if (is_k) {
                    const uint32_t tile = base + C::kOffRaw + st * C::kRaw + sub0 * T::kTileBytes;
                    const int there = static_cast<int>((note >> (8 * sub0)) & 255u);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // tokens 8 h + g
                        uint32_t pr[G], sc[G], mn[G];
                        lds_params<G>(tile + T::kKParams + (8 * h + g) * G * 4, pr);
                        if (there < 16) {
#pragma unroll
                            for (int y = 0; y < G; ++y)
                                if (8 * h + g >= there) pr[y] = 0;
                        }
#pragma unroll
                        for (int y = 0; y < G; ++y) {
                            sc[y] = __byte_perm(pr[y], 0, 0x1010);
                            mn[y] = __byte_perm(pr[y], 0, 0x3232);
                        }
                        auto put = [&](int y, int w, uint32_t word) {
                            uint32_t q[4];
                            codes(word, q);
#pragma unroll
                            for (int x = 0; x < 4; ++x) q[x] = hfma2(q[x], sc[y], mn[y]);
                            sts128(to_k + h * 1024 + y * (C::kTokCta * 128) + (((2 * t + w) ^ g) << 4), q[0], q[1], q[2], q[3]);
                        };
                        if constexpr (G == 1) {
                            const uint2 v = lds64(tile + (h * 32 + lane) * 8);
                            put(0, 0, v.x);
                            put(0, 1, v.y);
                        } else {
#pragma unroll
                            for (int j = 0; j < G / 2; ++j) {
                                const uint4 v = lds128(tile + ((2 * j + h) * 32 + lane) * 16);
                                put(2 * j, 0, v.x);
                                put(2 * j, 1, v.y);
                                put(2 * j + 1, 0, v.z);
                                put(2 * j + 1, 1, v.w);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int vs = 0; vs < kValues; ++vs) {
                        const uint32_t tile = base + C::kOffRaw + st * C::kRaw + (sub0 + vs) * T::kTileBytes;
                        const uint32_t to_v = (vs == 0 ? to_v0 : to_v1) + buf * C::kBuf;
                        const int there = static_cast<int>((note >> (8 * (sub0 + vs))) & 255u);
                        // groups y0 .. of the V codes, words x0 .. of each (heads of 64 have one group: half of its words)
                        constexpr int kY = G == 1 ? 1 : G / C::kCtas, kX = Pair && G == 1 ? 2 : 4;
                        const int y0 = G == 1 ? 0 : static_cast<int>(rank) * kY;
                        uint32_t pr[4][kY];  // tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int token = 2 * t + (k & 1) + 8 * (k >> 1);
                            lds_params<kY>(tile + T::kVParams + token * G * 4 + y0 * 4, pr[k]);
                            if (there < 16 && token >= there) {
#pragma unroll
                                for (int y = 0; y < kY; ++y) pr[k][y] = 0;
                            }
                        }
#pragma unroll
                        for (int y = 0; y < kY; ++y) {
                            const uint32_t sa = __byte_perm(pr[0][y], pr[1][y], 0x5410), ma = __byte_perm(pr[0][y], pr[1][y], 0x7632);
                            const uint32_t sb = __byte_perm(pr[2][y], pr[3][y], 0x5410), mb = __byte_perm(pr[2][y], pr[3][y], 0x7632);
                            uint32_t w[4];
                            if constexpr (kX == 4) {
                                const uint4 v = lds128(tile + T::kV + (y0 + y) * 512 + lane * 16);
                                w[0] = v.x;
                                w[1] = v.y;
                                w[2] = v.z;
                                w[3] = v.w;
                            } else {
                                const uint2 v = lds64(tile + T::kV + lane * 16 + rank * 8);
                                w[0] = v.x;
                                w[1] = v.y;
                            }
#pragma unroll
                            for (int x = 0; x < kX; ++x) {
                                uint32_t q[4];
                                codes(w[x], q);
                                stmatrix4(to_v + (64 * y + 16 * x) * 128, hfma2(q[0], sa, ma), hfma2(q[1], sa, ma), hfma2(q[2], sb, mb),
                                          hfma2(q[3], sb, mb));
                            }
                        }
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(is_k ? k_full(buf) : v_full(buf));
                    mbar_arrive(raw_empty(st));
                }
            }
        } else if (warp == kProducer) {
            // ================= fetch: four 16-token tiles a stage, page numbers of 8 stages at a time
            const uint64_t policy = policy_evict_last();
            int64_t from = -1;
            int there = 0;
            for (int i = 0; i < nt; ++i) {
                const uint32_t it = done + i, st = it % R;
                if ((i & 7) == 0) {
                    const int64_t tok = static_cast<int64_t>(t0 + i) * kTok + lane * kKv4Tile;
                    there = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(kKv4Tile), sq.n - tok)));
                    from = -1;
                    if (there > 0 && i + lane / kSub < nt && in_bounds((tok >> cache.page_shift) < p.max_pages, status)) {
                        const int page = p.block_table[static_cast<int64_t>(b) * p.max_pages + (tok >> cache.page_shift)];
                        if (page >= 0 && page < cache.num_pages) {
                            from = cache.tile_offset<D>(page, kvh, static_cast<int>(tok) & ((1 << cache.page_shift) - 1));
                            if (!in_bounds(from >= 0 && from + T::kTileBytes <= cache.bytes<D>(), status)) from = -1;
                        } else {
                            record_error(status, kErrBounds);
                        }
                    }
                }
                if (!wait(raw_empty(st), ((it / R) & 1) ^ 1)) break;
                const bool mine = lane / kSub == (i & 7) && from >= 0;
                const uint32_t have = __ballot_sync(0xffffffffu, mine);
                uint32_t note = lane / kSub == (i & 7) && from >= 0 ? static_cast<uint32_t>(there) << (8 * (lane % kSub)) : 0u;
                note = __reduce_or_sync(0xffffffffu, note);
                if (lane == 0) {
                    s_valid[it % kNotes] = note;
                    mbar_arrive_expect_tx(raw_full(st), static_cast<uint32_t>(__popc(have)) * T::kTileBytes);
                }
                __syncwarp();
                if (mine && (!kDebugBounds || static_cast<int>(it) != p.withhold))
                    bulk_g2s(base + C::kOffRaw + st * C::kRaw + (lane % kSub) * T::kTileBytes, cache.pages + from, T::kTileBytes,
                             raw_full(st), policy);
                issued = it + 1;
            }
        } else if (warp == kIssueS) {
            // ================= S = Q . K'^T
            constexpr uint32_t idesc = idesc_f16_f32(C::kUnitRows, kTok);
            if constexpr (Pair)
                for (int i = 0; i < nt && rank != 0 && pass_on(k_full((done + i) % KB), (done + i) / KB & 1); ++i) {
                }
            bool ok = rank == 0 && wait_all(q_full, segment & 1);
            for (int i = 0; i < nt && ok; ++i) {
                const uint32_t it = done + i, buf = it & 1, use = it >> 1, kb = it % KB;
                ok = wait_all(k_full(kb), it / KB & 1) && wait(pv_done(buf), (use & 1) ^ 1);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t desc = smem_desc_sw128(base + kb * C::kBuf + (k / 4) * (C::kTokCta * 128)) + (k & 3) * 2;
                        multiply(tmem + C::kColS + buf * kTok, tmem + C::kColQ + 8 * k, desc, idesc, k > 0);
                    }
                    commit(s_full(buf));
                    if constexpr (KB > 2) commit(k_free(kb));
                }
                __syncwarp();
            }
        } else {
            // ================= O += P . V'
            constexpr uint32_t idesc = idesc_f16_f32(C::kUnitRows, D);
            if constexpr (Pair)
                for (int i = 0; i < nt && rank != 0 && pass_on(v_full((done + i) % KB), (done + i) / KB & 1); ++i) {
                }
            for (int i = 0; i < nt && rank == 0; ++i) {
                const uint32_t it = done + i, buf = it & 1, use = it >> 1, kb = it % KB;
                if (!wait_all(v_full(kb), it / KB & 1) || !wait_all(p_full(buf), use & 1)) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kTok / 16; ++k) {
                        const uint64_t desc = smem_desc_sw128(base + C::kOffV + kb * C::kBuf) + k * 2;
                        multiply(tmem, tmem + C::kColS + buf * kTok + 8 * k, desc, idesc, i > 0 || k > 0);
                    }
                    commit(pv_done(buf));
                    if constexpr (KB > 2) commit(v_free(kb));
                }
                __syncwarp();
            }
        }
        done += nt;
        ++segment;

        if (parts > kJoinInPlace) {
            // ---- more parts than that: all threads of the last CTA add them from memory, in the same order
            __syncthreads();
            if (*s_last && !*s_abort && rows > 0) {
                __threadfence();
                // What each part's rows are scaled by: kGroups groups of threads (6, of a pair 5), every kGroups-th
                // part each. (K' and V' are not in use: all their products are done.)
                constexpr int kGroups = kThreads / kRows;
                const int n = parts;
                float* s_f = reinterpret_cast<float*>(smem);  // [n][128]
                // 8 elements of a row a thread, from four parts in one round of loads (the first one's before
                // the factors are known)
                const int items = rows * (D / 8);
                float4 a[4][2];
                auto load = [&](int x, int c) {
                    const int c8 = x / rows, r = x - c8 * rows;
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const float4* from = reinterpret_cast<const float4*>(part_of(cta0, cta0 + C::kCtas * min(c + h, n - 1)) + 2 * kRows) + r;
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            a[h][k] = x < items && c + h < n ? __ldcg(from + (2 * c8 + k) * kRows) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                };
                load(tid, 0);
                {
                    const int grp = tid / kRows, r = min(tid & (kRows - 1), rows - 1);
                    float top = -INFINITY;
                    if (grp < kGroups) {
                        for (int c = grp; c < n; c += kGroups) {
                            const float m = __ldcg(part_of(cta0, cta0 + C::kCtas * c) + r);
                            s_f[c * kRows + (tid & (kRows - 1))] = m;
                            top = fmaxf(top, m);
                        }
                        s_join[tid] = top;
                    }
                    __syncthreads();
                    if (grp < kGroups) {
                        for (int i = 0; i < kGroups; ++i) top = fmaxf(top, s_join[i * kRows + (tid & (kRows - 1))]);
                        for (int c = grp; c < n; c += kGroups) {
                            const float m = s_f[c * kRows + (tid & (kRows - 1))];
                            const float f = m == -INFINITY ? 0.f : ex2(m - top);
                            s_f[c * kRows + (tid & (kRows - 1))] = f;
                        }
                    }
                    __syncthreads();
                    if (tid < kRows) {
                        float total = 0.f;
                        for (int c = 0; c < n; c += 4) {
                            float l[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) l[k] = c + k < n ? __ldcg(part_of(cta0, cta0 + C::kCtas * (c + k)) + kRows + r) : 0.f;
#pragma unroll
                            for (int k = 0; k < 4; ++k) total = c + k < n ? fmaf(l[k], s_f[(c + k) * kRows + tid], total) : total;
                        }
                        s_join[kJoinInPlace * kRows + tid] = total > 0.f ? 1.f / total : 0.f;
                        if (p.lse != nullptr && tid < rows) {
                            const int in_seq = row0 + tid, pos = in_seq / sq.grp, hd = in_seq - pos * sq.grp;
                            p.lse[static_cast<int64_t>(sq.q0 + pos) * p.heads + kvh * sq.grp + hd] =
                                total > 0.f ? 0.6931471805599453f * (top - kLift + log2f(total)) : -INFINITY;
                        }
                    }
                    __syncthreads();
                }
                for (int x = tid; x < items; x += kThreads) {
                    const int c8 = x / rows, r = x - c8 * rows;
                    float4 v[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
                    for (int c = 0; c < n; c += 4) {
                        if (x != tid || c != 0) load(x, c);
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const float f = c + h < n ? s_f[(c + h) * kRows + r] : 0.f;
                            if (f == 0.f) continue;  // (a part that saw nothing may hold anything)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                v[k].x = fmaf(a[h][k].x, f, v[k].x);
                                v[k].y = fmaf(a[h][k].y, f, v[k].y);
                                v[k].z = fmaf(a[h][k].z, f, v[k].z);
                                v[k].w = fmaf(a[h][k].w, f, v[k].w);
                            }
                        }
                    }
                    const int in_seq = row0 + r, pos = in_seq / sq.grp, hd = in_seq - pos * sq.grp;
                    const int64_t at_out = static_cast<int64_t>(sq.q0 + pos) * p.heads + kvh * sq.grp + hd;
                    const float inv = s_join[kJoinInPlace * kRows + r];
                    const __half2 h0 = __floats2half2_rn(v[0].x * inv, v[0].y * inv), h1 = __floats2half2_rn(v[0].z * inv, v[0].w * inv);
                    const __half2 h2 = __floats2half2_rn(v[1].x * inv, v[1].y * inv), h3 = __floats2half2_rn(v[1].z * inv, v[1].w * inv);
                    *reinterpret_cast<uint4*>(p.out + at_out * D + 8 * c8) =
                        make_uint4(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1),
                                   *reinterpret_cast<const uint32_t*>(&h2), *reinterpret_cast<const uint32_t*>(&h3));
                }
            }
        }
        // Q, O and the barriers' phases belong to the next segment from here on (all threads leave, or none)
        if (__syncthreads_or(*static_cast<volatile int*>(s_abort))) break;
    }
    if (*s_abort) {  // what is under way ends before the memory is given back (bounded)
        if (warp == kProducer) {
            for (uint32_t it = issued < R ? 0 : issued - R; it < issued; ++it)
                for (int n = 0; n < 65536 && !mbar_test_wait(raw_full(it % R), (it / R) & 1); ++n) {
                }
        } else if (warp >= kIssueS) {
            const uint32_t bar = drained(warp - kIssueS);
            if (rank == 0 && elect_one()) commit(bar);
            for (int n = 0; n < 65536 && !mbar_test_wait(bar, 0); ++n) {
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    if constexpr (Pair) cluster_sync_all();  // (the other's products read this one's memory)
    else __syncthreads();
    tc_fence_after();
    if (warp == kProducer) {
        if constexpr (Pair) tmem_pair_dealloc(tmem, C::kCols);
        else tmem_dealloc(tmem, C::kCols);
    }
}

template <int D, bool Pair>
cudaError_t launch_prompt(const Kv4AttnParams& p, const Kv4View& v, const LaunchCtx& ctx) {
    using C = Prompt<D, Pair>;
    cudaError_t e = cudaFuncSetAttribute(kv4_prompt_kernel<D, Pair>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min(ctx.sm_count, kKv4MaxPromptCtas) / C::kCtas * C::kCtas), 1, 1);
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C::kCtas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = Pair ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kv4_prompt_kernel<D, Pair>, p, v, ctx.timeout_ns, ctx.status);
}

}  // namespace

size_t kv4_prompt_workspace(int head_dim) {
    return 4096 + static_cast<size_t>(2 * kKv4MaxPromptCtas) * kRows * (head_dim + 2) * 4;
}

// Two CTAs on 256 rows save 4 to 14 % of what one on 128 twice takes, and are worth no less for a half-empty last
// unit: an even number of 128-row units a sequence (one sequence of 4096, heads of 256, 4096 queries of 5 heads a key
// head: 189.9 us with one, 182.1 with two; 8 of 4096, 240 rows 48.3 | 45.7, heads of 64 95.1 | 91.4), or so many that
// the last does not count, 3 of heads of 256 and 17 of others (300 rows, heads of 256: 36.0 | 33.1 one sequence, 63.4 |
// 64.6 eight; of 128 81.7 | 95.8, of 64 136.2 | 169.2). So pairs may take a third, or a 17th, more CTAs for the whole
// batch. (A prompt of 512 queries among 15 or 63 streams of one, all of 4096 tokens, 4 heads of 256: 79.1 | 96.6, 171.3
// | 249.9.)
bool kv4_prompt_pairs(const Kv4AttnParams& p, int kv_heads, int head_dim) {
    const int64_t units = kv4_row_groups(p, kv_heads, kRows), ctas = 2 * kv4_row_groups(p, kv_heads, 2 * kRows);
    return head_dim == 256 ? 3 * ctas <= 4 * units : 17 * ctas <= 18 * units;
}

cudaError_t launch_kv4_prompt(const Kv4AttnParams& p, const Kv4View& v, int head_dim, bool pair, const LaunchCtx& ctx) {
    switch (head_dim) {
        case 64: return pair ? launch_prompt<64, true>(p, v, ctx) : launch_prompt<64, false>(p, v, ctx);
        case 128: return pair ? launch_prompt<128, true>(p, v, ctx) : launch_prompt<128, false>(p, v, ctx);
        default: return pair ? launch_prompt<256, true>(p, v, ctx) : launch_prompt<256, false>(p, v, ctx);
    }
}

}  // namespace w4a16
