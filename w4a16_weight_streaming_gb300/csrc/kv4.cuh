// The 4-bit paged key/value cache: device-side addressing and scalar decoding, shared by the append,
// load and attention kernels.
//
// A page holds `page_tokens` (a power of two, >= 16) tokens of every key/value head; the tokens of one
// head of one page are one contiguous run of 16-token tiles. A tile of head size D (18 D bytes,
// a multiple of 128) is everything 16 tokens of one head need, so one bulk copy fetches it:
//   [K codes 8 D][V codes 8 D][K parameters 16 x D/64 x 4][V parameters 16 x D/64 x 4]
// A parameter is the fp16 pair (scale, min) of 64 consecutive elements: x' = min + code * scale.
// The codes lie in the order in which the m16n8k16 matrix instruction wants its A operand, lane
// l = 4 g + t (g = l / 4, t = l % 4), so that a lane's registers come from vector loads and two
// instructions a pair, without any exchange between lanes:
//   K codes (A = 16 tokens x 16 elements). Token h * 8 + g, element 64 y + 16 t + 8 w + i: word w of the
//     8 bytes that lane (g, t) holds of (half h, group y); two groups side by side make the lane's 16
//     bytes (D = 64 has one group, 8 bytes a lane). Nibble i/2 + 4 (i & 1) of the word.
//   V codes (A = 16 elements x 16 tokens). Element 64 y + 16 i + 8 u + g: byte of word i of the 16 bytes
//     that lane (g, t) holds of group y; token k: t = (k & 7) / 2, byte 2 (k & 1) + k / 8, nibble u. So
//     no two tokens share a byte, and tokens may be stored in any order without read-modify-write.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace w4a16 {

#ifdef W4A16_DEBUG_BOUNDS
constexpr bool kDebugBounds = true;
#else
constexpr bool kDebugBounds = false;
#endif

constexpr int kKv4Group = 64;  // elements per (scale, min) pair
constexpr int kKv4Tile = 16;   // tokens per tile

template <int D>
struct Kv4 {
    static constexpr int kGroups = D / kKv4Group;
    static constexpr int kCodes = kKv4Tile * D / 2;               // bytes of one tile's K (or V) codes
    static constexpr int kParams = kKv4Tile * kGroups * 4;        // bytes of one tile's K (or V) parameters
    static constexpr int kV = kCodes;                             // offsets inside a tile
    static constexpr int kKParams = 2 * kCodes;
    static constexpr int kVParams = 2 * kCodes + kParams;
    static constexpr int kTileBytes = 2 * kCodes + 2 * kParams;   // 18 D

    // Byte offset of the K word of elements d .. d+7 (d % 8 == 0) of token k.
    __device__ static __forceinline__ int k_word(int k, int d) {
        const int h = k >> 3, g = k & 7, y = d >> 6, t = (d >> 4) & 3, w = (d >> 3) & 1;
        if (D == 64) return (h * 32 + g * 4 + t) * 8 + w * 4;
        return (((y >> 1) * 2 + h) * 32 + g * 4 + t) * 16 + (y & 1) * 8 + w * 4;
    }
    // Byte offset (from the tile's start) of the V codes of token k, elements 16 j + g (low nibble) and
    // 16 j + 8 + g (high nibble).
    __device__ static __forceinline__ int v_byte(int k, int j, int g) {
        return kV + (j >> 2) * 512 + (g * 4 + ((k & 7) >> 1)) * 16 + (j & 3) * 4 + ((k & 1) << 1) + (k >> 3);
    }
    __device__ static __forceinline__ int k_param(int k, int y) { return kKParams + (k * kGroups + y) * 4; }
    __device__ static __forceinline__ int v_param(int k, int y) { return kVParams + (k * kGroups + y) * 4; }
};

// The cache as the kernels see it.
struct Kv4View {
    uint8_t* pages;
    int num_pages;
    int page_shift;  // log2(page_tokens)
    int kv_heads;

    __device__ __forceinline__ int64_t slots() const { return static_cast<int64_t>(num_pages) << page_shift; }
    // Byte offset of the tile that holds token `in_page` of head `head` of page `page`.
    template <int D>
    __device__ __forceinline__ int64_t tile_offset(int page, int head, int in_page) const {
        const int64_t run = static_cast<int64_t>(page) * kv_heads + head;
        return ((run << (page_shift - 4)) + (in_page >> 4)) * Kv4<D>::kTileBytes;
    }
    template <int D>
    __device__ __forceinline__ int64_t bytes() const {
        return (static_cast<int64_t>(num_pages) * kv_heads << (page_shift - 4)) * Kv4<D>::kTileBytes;
    }
};

// Warp-wide bounded wait of the kv4 kernels: the hardware's suspending test, so that a waiting warp leaves
// its issue slots to the others. (27 warps that polled with test_wait took 283 us for a prompt chunk of
// 1024 x 20 heads behind 8192 tokens, with pauses of 20 to 200 ns between two looks 190, suspended 177.)
__device__ __forceinline__ bool warp_suspend(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t timeout_ns,
                                             unsigned* status) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t spin = 1;; ++spin) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        bool over = *abort_flag != 0;
        if (!over && (spin & 31u) == 0u && global_timer_ns() - t0 > timeout_ns) {
            record_error(status, kErrTimeout);
            *abort_flag = 1;
            over = true;
        }
        if (__any_sync(0xffffffffu, over)) return false;
    }
}

// Wait for arrivals of the other CTA too (a suspended thread is not woken promptly by those: polled).
__device__ __forceinline__ bool warp_poll_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t timeout_ns,
                                                  unsigned* status) {
    if (__all_sync(0xffffffffu, mbar_test_wait_cluster(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t spin = 1;; ++spin) {
        if (__all_sync(0xffffffffu, mbar_test_wait_cluster(bar, parity))) return true;
        if ((spin & 255u) != 0u) continue;
        bool over = *abort_flag != 0;
        if (!over && global_timer_ns() - t0 > timeout_ns) {
            record_error(status, kErrTimeout);
            *abort_flag = 1;
            over = true;
        }
        if (__any_sync(0xffffffffu, over)) return false;
    }
}

// ---- kv4_prompt.cu: the tcgen05 kernel for many query rows a sequence.
struct Kv4AttnParams;
struct LaunchCtx;
constexpr int kKv4MaxPromptCtas = 160;
size_t kv4_prompt_workspace(int head_dim);
bool kv4_prompt_pairs(const Kv4AttnParams& p, int kv_heads, int head_dim);
cudaError_t launch_kv4_prompt(const Kv4AttnParams& p, const Kv4View& v, int head_dim, bool pair, const LaunchCtx& ctx);

}  // namespace w4a16
