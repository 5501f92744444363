// attnres_cache.cu -- writing source rows into the compressed cache and
// reading them back (record layout: cached.cuh).
//
// Write: x = v * 2^k with k the smallest exponent for which the group's
// largest magnitude is at most the format's largest (448 = 1.75 * 2^8 for
// e4m3, 6 = 1.5 * 2^2 for e2m1), so no code saturates; dividing by 2^k is
// exact and the codes are rounded to nearest, ties to even.  k comes from the
// bf16 bits of the group's largest magnitude (integer maximum: a NaN or an
// infinity is the largest of all).  The mean square of the key channels'
// decoded values is summed in FP32 in a fixed order.
#include "cached.cuh"
#include "kernels.cuh"
#include "launch_pdl.cuh"

namespace attnres {
namespace {

__device__ unsigned g_cache_error;

constexpr int kRowWarps = 4;  // warps per CTA

// Largest |x| of a 16-byte vector as bf16 bits in each half of a word.
__device__ __forceinline__ uint32_t abs_max8(const uint4& v) {
    const uint32_t m = 0x7fff7fffu;
    return __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
}

template <int BITS>
__global__ void __launch_bounds__(kRowWarps * 32) cache_write_kernel(const CacheRowsArgs a) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long stride = static_cast<long long>(gridDim.x) * kRowWarps;
    for (long long n = static_cast<long long>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5); n < a.N; n += stride) {
        const uint16_t* x = a.x + n * a.x_ld;
        unsigned char* row = a.rows + n * a.row_ld;
        const int padded = static_cast<int>(a.codes) * 8 / BITS;  // channels the code area holds
        float sq = 0.0f;
        for (int base = 0; base < padded; base += 256) {  // 8 channels a lane, 4 lanes a group
            const int c = base + lane * 8;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (c < a.D) v = ld_global_nc_v4(x + c);
            const uint32_t m2 = abs_max8(v);
            uint32_t m = max(m2 & 0xffffu, m2 >> 16);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const bool finite = m < 0x7f80u;
            float f[8];
            unpack8(v, f);
            if (m > kCacheClip) {  // rare: magnitudes next to the float range's end, NaN, infinity
                const float lim = bf16_bits_to_float(kCacheClip);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = finite ? fminf(fmaxf(f[i], -lim), lim) : 0.0f;
                m = kCacheClip;
            }
            const int e = static_cast<int>(m >> 7), mant = static_cast<int>(m & 0x7fu);
            int k = BITS == 8 ? e - 135 + (mant > 0x60) : e - 129 + (mant > 0x40);
            k = max(k, kCacheMinExp);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
            uint32_t h[4];  // the codes' values as half pairs
            if constexpr (BITS == 8) {
                uint32_t w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
                        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
                        : "=r"(w[i])
                        : "f"(f[4 * i] * down), "f"(f[4 * i + 1] * down), "f"(f[4 * i + 2] * down),
                          "f"(f[4 * i + 3] * down));
                    cache_unpack8(w[i], h[2 * i], h[2 * i + 1]);
                }
                if (c < padded) *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
            } else {
                uint32_t w;
                asm("{\n\t.reg .b8 e, f, g, h;\n\tcvt.rn.satfinite.e2m1x2.f32 e, %2, %1;\n\t"
                    "cvt.rn.satfinite.e2m1x2.f32 f, %4, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 g, %6, %5;\n\t"
                    "cvt.rn.satfinite.e2m1x2.f32 h, %8, %7;\n\tmov.b32 %0, {e, f, g, h};\n\t}"
                    : "=r"(w)
                    : "f"(f[0] * down), "f"(f[1] * down), "f"(f[2] * down), "f"(f[3] * down), "f"(f[4] * down),
                      "f"(f[5] * down), "f"(f[6] * down), "f"(f[7] * down));
                cache_unpack4(w, h[0], h[1], h[2], h[3]);
                if (c < padded) *reinterpret_cast<uint32_t*>(row + c / 2) = w;
            }
            if ((lane & 3) == 0 && c < a.D) row[a.codes + c / 32] = finite ? static_cast<uint8_t>(k + 127) : 255;
            float g0 = 0.0f, g1 = 0.0f;
            const bool any = c < a.ko + a.R && c + 8 > a.ko;
            if (any) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = c + 2 * i;
                    uint32_t hm = h[i];
                    if (j < a.ko || j >= a.ko + a.R) hm &= 0xffff0000u;
                    if (j + 1 < a.ko || j + 1 >= a.ko + a.R) hm &= 0x0000ffffu;
                    half2_dot(hm, hm, g0, g1);
                }
                sq += finite ? (g0 + g1) * up * up : __uint_as_float(0x7fc00000u);
            }
        }
        sq = warp_sum(sq);
        if (lane == 0)
            *reinterpret_cast<uint2*>(row + a.stat) = make_uint2(__float_as_uint(sq / static_cast<float>(a.R)), a.tag);
        // bytes between the scales and the statistic, and behind the tag
        const uint32_t g = static_cast<uint32_t>(a.D + 31) / 32;
        for (uint32_t b = a.codes + g + lane; b < a.stat; b += 32) row[b] = 0;
        if (((a.stat + 8) & 15u) && lane == 0) *reinterpret_cast<uint2*>(row + a.stat + 8) = make_uint2(0u, 0u);
    }
}

// One thread decodes 8 channels; a record that is not one in this format
// reads as NaN and is recorded.
template <int BITS>
__global__ void __launch_bounds__(256) cache_load_kernel(const CacheRowsArgs a) {
    pdl_wait();
    const uint32_t per_row = static_cast<uint32_t>(a.D) / 8u;
    const long long total = a.N * per_row;
    const long long stride = static_cast<long long>(gridDim.x) * 256;
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < total; i += stride) {
        const long long n = i / per_row;
        const uint32_t c = static_cast<uint32_t>(i - n * per_row) * 8u;
        const unsigned char* row = a.rows + n * a.row_ld;
        uint32_t h[4];
        if constexpr (BITS == 8) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(row + c));
            cache_unpack8(w.x, h[0], h[1]);
            cache_unpack8(w.y, h[2], h[3]);
        } else {
            cache_unpack4(__ldg(reinterpret_cast<const uint32_t*>(row + c / 2)), h[0], h[1], h[2], h[3]);
        }
        float up = cache_scale(__ldg(row + a.codes + c / 32));
        const uint32_t tag = __ldg(reinterpret_cast<const uint32_t*>(row + a.stat + 4));
        if ((tag ^ a.tag) & kCacheTagFormat) {
            atomicCAS(&g_cache_error, 0u, kSiteCacheTag);
            up = __uint_as_float(0x7fc00000u);
        }
        uint4 o;
        const f2 s = f2_dup(up);
        o.x = f2_to_bf16(f2_mul(f2_half(h[0]), s));
        o.y = f2_to_bf16(f2_mul(f2_half(h[1]), s));
        o.z = f2_to_bf16(f2_mul(f2_half(h[2]), s));
        o.w = f2_to_bf16(f2_mul(f2_half(h[3]), s));
        *reinterpret_cast<uint4*>(a.out + n * a.x_ld + c) = o;
    }
}

int grid_for(long long blocks, int most) {
    return static_cast<int>(blocks < most ? (blocks < 1 ? 1 : blocks) : most);
}

}  // namespace

unsigned take_cache_rows_error() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_cache_error, sizeof v) != cudaSuccess) return 0xffffffffu;
    if (v) cudaMemcpyToSymbol(g_cache_error, &zero, sizeof zero);
    return v;
}

cudaError_t launch_cache_write(const CacheRowsArgs& a, int bits, int sm_count, cudaStream_t stream) {
    const int grid = grid_for((a.N + kRowWarps - 1) / kRowWarps, sm_count * 16);
    auto kern = bits == 8 ? cache_write_kernel<8> : cache_write_kernel<4>;
    return launch_pdl(kern, dim3(grid), dim3(kRowWarps * 32), 0, stream, a);
}

cudaError_t launch_cache_load(const CacheRowsArgs& a, int bits, int sm_count, cudaStream_t stream) {
    const int grid = grid_for((a.N * (a.D / 8) + 255) / 256, sm_count * 8);
    auto kern = bits == 8 ? cache_load_kernel<8> : cache_load_kernel<4>;
    return launch_pdl(kern, dim3(grid), dim3(256), 0, stream, a);
}

}  // namespace attnres
