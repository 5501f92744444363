// cached.cuh -- the compressed source cache: record layout, decoding, kernel
// arguments and launchers (internal to the library).
//
// One record per token and source, all parts in one run of memory:
//   codes   D channels: e4m3 bytes, or e2m1 nibbles (channel 2i in the low
//           half of byte i); zeros up to a multiple of 16 bytes
//   scales  one byte per 32 channels, the exponent k of 2^k plus 127; a
//           group that held a NaN or an infinity has 255 and zero codes.
//           Its scale decodes as +inf, and 0 * inf is the NaN it reads as
//   stat    float: mean square of the key channels' values (8-byte aligned)
//   tag     uint32: R | key_offset << 14 | (bits == 8) << 27 | 5 << 28, so
//           that a read with another key slice, or of memory that no write
//           filled, is noticed
//   pad     to a multiple of 16 bytes
#pragma once

#include <cstddef>
#include <cstdint>
#include <mutex>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attnres.h"
#include "device_utils.cuh"

namespace attnres {

constexpr int kCacheGroup = 32;          // channels per scale, and channels per thread of the read kernels
constexpr int kCacheMinExp = -110;       // smallest k: every value stays a normal float and bf16
constexpr unsigned kCacheClip = 0x7f40;  // bf16 1.5 * 2^127: larger magnitudes are held as it, since rounding
                                         // them to the format's few bits could leave the float range

__host__ __device__ constexpr uint32_t cache_code_bytes(int D, int bits) {
    return (static_cast<uint32_t>(D) * bits / 8 + 15u) & ~15u;
}
__host__ __device__ constexpr uint32_t cache_stat_offset(int D, int bits) {
    return cache_code_bytes(D, bits) + ((static_cast<uint32_t>(D + 31) / 32 + 7u) & ~7u);
}
__host__ __device__ constexpr uint32_t cache_row_bytes(int D, int bits) {
    return (cache_stat_offset(D, bits) + 8u + 15u) & ~15u;
}
__host__ __device__ constexpr uint32_t cache_tag(int R, int ko, int bits) {
    return static_cast<uint32_t>(R) | static_cast<uint32_t>(ko) << 14 | (bits == 8 ? 1u << 27 : 0u) | 5u << 28;
}
// The part of a tag that says the record is one, in this format.
constexpr uint32_t kCacheTagFormat = 0xf8000000u;

// 2^(byte - 127) (0 for byte 0, which no write makes; +inf for 255).
__device__ __forceinline__ float cache_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Four bytes of codes -> half pairs, exact: e4m3 and e2m1 values are halves.
__device__ __forceinline__ void cache_unpack8(uint32_t w, uint32_t& a, uint32_t& b) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(w));
}
__device__ __forceinline__ void cache_unpack4(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm("{\n\t.reg .b8 e, f, g, h;\n\tmov.b32 {e, f, g, h}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, e;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, f;\n\tcvt.rn.f16x2.e2m1x2 %2, g;\n\tcvt.rn.f16x2.e2m1x2 %3, h;\n\t}"
        : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
        : "r"(w));
}

// A pair of floats as one 64-bit register, so that it stays an aligned pair
// from one packed instruction to the next.
using f2 = unsigned long long;
__device__ __forceinline__ f2 f2_make(float x, float y) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ f2 f2_dup(float x) { return f2_make(x, x); }
__device__ __forceinline__ float2 f2_get(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ float f2_sum(f2 v) {
    const float2 r = f2_get(v);
    return r.x + r.y;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 f2_half(uint32_t h) {  // of a half pair, as half * 1 + 0
    f2 r;
    asm("{\n\t.reg .b16 l, h, one;\n\t.reg .f32 x, y;\n\tmov.b32 {l, h}, %1;\n\tmov.b16 one, 0x3c00;\n\t"
        "fma.rn.f32.f16 x, l, one, 0f00000000;\n\tfma.rn.f32.f16 y, h, one, 0f00000000;\n\tmov.b64 %0, {x, y};\n\t}"
        : "=l"(r)
        : "r"(h));
    return r;
}
__device__ __forceinline__ f2 f2_bf16(uint32_t w) {  // of a bf16 pair
    return f2_make(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t f2_to_bf16(f2 v) { return pack_f2(f2_get(v)); }

// s0 += a_lo * b_lo, s1 += a_hi * b_hi for half pairs (exact products, FP32 sums).
__device__ __forceinline__ void half2_dot(uint32_t a, uint32_t b, float& s0, float& s1) {
    asm("{\n\t.reg .b16 al, ah, bl, bh;\n\tmov.b32 {al, ah}, %2;\n\tmov.b32 {bl, bh}, %3;\n\t"
        "fma.rn.f32.f16 %0, al, bl, %0;\n\tfma.rn.f32.f16 %1, ah, bh, %1;\n\t}"
        : "+f"(s0), "+f"(s1)
        : "r"(a), "r"(b));
}

// The codes of one thread's 32 channels.
template <int BITS>
struct CacheCodes {
    uint32_t w[BITS];  // 4 words of nibbles or 8 words of bytes
    // half pairs of channels 2i, 2i + 1
    __device__ __forceinline__ void unpack(uint32_t (&h)[16]) const {
        if constexpr (BITS == 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) cache_unpack8(w[i], h[2 * i], h[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) cache_unpack4(w[i], h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
        }
    }
};

struct CacheRowsArgs {
    const uint16_t* x;  // write: source rows; load: NULL
    uint16_t* out;      // load: destination rows
    unsigned char* rows;
    long long N, x_ld, row_ld;
    int D, R, ko;
    uint32_t codes, stat;
    uint32_t tag;
};

// The read over cached rows and its gradient share the description of the sources.
struct CachedArgs {
    const unsigned char* rows[ATTNRES_MAX_S];
    long long N, row_ld, live_ld;
    int S, D, R, ko;  // S: cached sources (a live one, read last, is not counted)
    uint32_t codes, stat, tag;
    float eps, scale;
    const uint16_t* live;
    const uint16_t* q;
    const uint16_t* w_o;
    float* alpha;  // [N][S + live]; the backward reads them
    float* rstd;
    float* logit;
    float* o_rstd;
    uint16_t* y;
};

struct CachedBwdArgs {
    CachedArgs c;
    uint16_t* dsrc[ATTNRES_MAX_S];
    long long dsrc_ld, dlive_ld;
    int want_dsrc;
    int wide_src, wide_live;  // gradient rows start on 32-byte boundaries and D % 16 == 0
    int seg;                  // rows a segment (the launcher's)
    uint16_t* dlive;
    const uint16_t* dy;
    float* part;  // [grid][R + D with the output norm]
};

// Threads that share a token: one per 32 channels, a power of two up to a
// warp, whole warps above.
inline int cached_team(int D) {
    const int g = (D + kCacheGroup - 1) / kCacheGroup;
    if (g > 32) return (g + 31) / 32 * 32;
    int t = 1;
    while (t < g) t *= 2;
    return t;
}
inline int cached_block(int D) {
    const int t = cached_team(D);
    return t > 32 ? t : 128;
}

// Raises a kernel's dynamic shared memory limit to `smem`, once a device and
// size, and says how many of its CTAs share an SM (registers and memory).
template <auto Kernel>
inline cudaError_t kernel_fit(int block, size_t smem, int* fit) {
    struct Known {
        size_t limit;
        int block, fit;
        size_t smem;
    };
    static std::mutex lock;
    static Known known[64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    std::lock_guard<std::mutex> hold(lock);
    Known local{};
    Known& k = dev < 64 ? known[dev] : local;
    if (smem > k.limit) {
        err = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (err != cudaSuccess) return err;
        k.limit = smem;
    }
    if (k.block != block || k.smem != smem) {
        err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&k.fit, Kernel, block, smem);
        if (err != cudaSuccess) return err;
        k.block = block;
        k.smem = smem;
    }
    *fit = k.fit;
    return k.fit > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
}

cudaError_t launch_cache_write(const CacheRowsArgs& a, int bits, int sm_count, cudaStream_t stream);
cudaError_t launch_cache_load(const CacheRowsArgs& a, int bits, int sm_count, cudaStream_t stream);
cudaError_t launch_cached_fwd(const CachedArgs& a, int bits, int sm_count, cudaStream_t stream);
int cached_bwd_grid(int S, bool live, long long N, int D, int bits, int sm_count);
cudaError_t launch_cached_bwd(CachedBwdArgs& a, int bits, int grid, int sm_count, cudaStream_t stream);
unsigned take_cache_rows_error();
// many tokens of rows of more than 512 channels: a warp or two a token (attnres_cached_wide.cuh)
cudaError_t launch_cached_wide8(const CachedArgs& a, int sm_count, cudaStream_t stream);
cudaError_t launch_cached_wide4(const CachedArgs& a, int sm_count, cudaStream_t stream);
unsigned take_cached_wide8_error();
unsigned take_cached_wide4_error();
unsigned take_cached_fwd_error();
unsigned take_cached_bwd_error();

}  // namespace attnres
