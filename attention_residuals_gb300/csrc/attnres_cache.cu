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
//
// A lane takes 8 channels a load (16 bytes), so the group's maximum is two
// shuffles.  What bounds the write: instructions and HBM together.  81920 rows
// of D=4096 under counters: 170 us in 8 bits (6.0 TB/s, 0.67 of the issue
// slots), 156 us in 4 (5.4 TB/s, 0.73).
//
// Load: v = code * 2^k, exact in bf16; 16 channels a lane.  HBM bounds it: nine
// sources of 8192 x 4096 from 4 bits in 119 us, 0.95 of the copy rate.
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

// One lane's 8 channels of a row: their codes to `row`, the group's scale byte
// returned, the sum of squares of the key channels among them added to `sq`.
template <int BITS>
__device__ __forceinline__ uint32_t quantise8(const CacheRowsArgs& a, unsigned char* row, int c, bool store, const uint4& v,
                                              float& sq) {
    const uint32_t m2 = abs_max8(v);
    uint32_t m = max(m2 & 0xffffu, m2 >> 16);  // over the four lanes of the group
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
                : "f"(f[4 * i] * down), "f"(f[4 * i + 1] * down), "f"(f[4 * i + 2] * down), "f"(f[4 * i + 3] * down));
            cache_unpack8(w[i], h[2 * i], h[2 * i + 1]);
        }
        if (store) *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
    } else {
        uint32_t w;
        asm("{\n\t.reg .b8 e, f, g, h;\n\tcvt.rn.satfinite.e2m1x2.f32 e, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 f, %4, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 g, %6, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 h, %8, %7;\n\tmov.b32 %0, {e, f, g, h};\n\t}"
            : "=r"(w)
            : "f"(f[0] * down), "f"(f[1] * down), "f"(f[2] * down), "f"(f[3] * down), "f"(f[4] * down), "f"(f[5] * down),
              "f"(f[6] * down), "f"(f[7] * down));
        cache_unpack4(w, h[0], h[1], h[2], h[3]);
        if (store) *reinterpret_cast<uint32_t*>(row + c / 2) = w;
    }
    if (c < a.ko + a.R && c + 8 > a.ko) {
        float g0 = 0.0f, g1 = 0.0f;
        if (c < a.ko || c + 8 > a.ko + a.R) {  // the key begins or ends among the lane's channels
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = c + 2 * i - a.ko;
                if (j < 0 || j >= a.R) h[i] &= 0xffff0000u;
                if (j + 1 < 0 || j + 1 >= a.R) h[i] &= 0x0000ffffu;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) half2_dot(h[i], h[i], g0, g1);
        sq += finite ? (g0 + g1) * up * up : __uint_as_float(0x7fc00000u);
    }
    return finite ? static_cast<uint32_t>(k + 127) : 255u;
}

// A warp (JOIN false) or a CTA (JOIN) writes a row: blocks of 256 U channels, 8
// a lane in each of U loads that are in flight together, four lanes a group.
// The scales of a block are stored by one instruction.
template <int BITS, int U, bool JOIN>
__global__ void __launch_bounds__(kRowWarps * 32) cache_write_kernel(const CacheRowsArgs a) {
    __shared__ float part[kRowWarps];
    pdl_wait();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int padded = static_cast<int>(a.codes) * 8 / BITS;  // channels the code area holds
    const uint32_t groups = static_cast<uint32_t>(a.D + 31) / 32;
    const long long stride = JOIN ? gridDim.x : static_cast<long long>(gridDim.x) * kRowWarps;
    for (long long n = JOIN ? blockIdx.x : static_cast<long long>(blockIdx.x) * kRowWarps + wid; n < a.N; n += stride) {
        const uint16_t* x = a.x + n * a.x_ld;
        unsigned char* row = a.rows + n * a.row_ld;
        float sq = 0.0f;
        for (int base = JOIN ? wid * 256 * U : 0; base < padded; base += JOIN ? kRowWarps * 256 * U : 256 * U) {
            uint4 v[U];
            uint32_t k[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = base + 256 * u + lane * 8;
                v[u] = c < a.D ? ld_global_nc_v4(x + c) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = base + 256 * u + lane * 8;
                k[u] = quantise8<BITS>(a, row, c, c < padded, v[u], sq);
            }
            // lane l stores the scale of the block's group l: load l / 8, lanes 4 (l % 8) ff.
            uint32_t mine = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t from = __shfl_sync(0xffffffffu, k[u], (lane & 7) * 4);
                if (lane >> 3 == u) mine = from;
            }
            const uint32_t g = static_cast<uint32_t>(base) / 32 + lane;
            if (lane < 8 * U && g < groups) row[a.codes + g] = static_cast<uint8_t>(mine);
        }
        sq = warp_sum(sq);
        if constexpr (JOIN) {
            if (lane == 0) part[wid] = sq;
            __syncthreads();
            sq = 0.0f;
#pragma unroll
            for (int u = 0; u < kRowWarps; ++u) sq += part[u];
            __syncthreads();
            if (wid != 0) continue;
        }
        if (lane == 0)
            *reinterpret_cast<uint2*>(row + a.stat) = make_uint2(__float_as_uint(sq / static_cast<float>(a.R)), a.tag);
        // bytes between the scales and the statistic, and behind the tag
        if (a.codes + groups + lane < a.stat) row[a.codes + groups + lane] = 0;
        if (((a.stat + 8) & 15u) && lane == 0) *reinterpret_cast<uint2*>(row + a.stat + 8) = make_uint2(0u, 0u);
    }
}

// 2^shift lanes read a row back, 16 channels each at a time; a record that is
// not one in this format reads as NaN and is recorded.
template <int BITS>
__global__ void __launch_bounds__(256) cache_load_kernel(const CacheRowsArgs a, int shift, int wide) {
    pdl_wait();
    const int per = 1 << shift, l = threadIdx.x & (per - 1);
    const long long stride = (static_cast<long long>(gridDim.x) * 256) >> shift;
    for (long long n = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) >> shift; n < a.N; n += stride) {
        const unsigned char* row = a.rows + n * a.row_ld;
        const uint32_t tag = __ldg(reinterpret_cast<const uint32_t*>(row + a.stat + 4));
        const bool good = !((tag ^ a.tag) & kCacheTagFormat);
        if (!good && l == 0) atomicCAS(&g_cache_error, 0u, static_cast<unsigned>(kSiteCacheTag));
#pragma unroll 4
        for (int c = l * 16; c < a.D; c += per * 16) {
            uint32_t h[8];
            if constexpr (BITS == 8) {
                const uint4 w = ld_global_nc_v4(row + c);
                cache_unpack8(w.x, h[0], h[1]);
                cache_unpack8(w.y, h[2], h[3]);
                cache_unpack8(w.z, h[4], h[5]);
                cache_unpack8(w.w, h[6], h[7]);
            } else {
                const uint2 w = __ldg(reinterpret_cast<const uint2*>(row + c / 2));
                cache_unpack4(w.x, h[0], h[1], h[2], h[3]);
                cache_unpack4(w.y, h[4], h[5], h[6], h[7]);
            }
            const float up = good ? cache_scale(__ldg(row + a.codes + c / 32)) : __uint_as_float(0x7fc00000u);
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = f2_to_bf16(f2_mul(f2_half(h[i]), f2_dup(up)));
            uint16_t* p = a.out + n * a.x_ld + c;
            if (wide) {
                asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                             "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                             : "memory");
            } else {
                st_global_cs_v4(p, make_uint4(o[0], o[1], o[2], o[3]));
                if (c + 8 < a.D) st_global_cs_v4(p + 8, make_uint4(o[4], o[5], o[6], o[7]));
            }
        }
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
    // Few wide rows: a CTA a row, so that a row's loads are all in flight at
    // once.  More rows than warps on the card have enough in flight.
    const bool join = a.D > 1024 && a.N <= static_cast<long long>(sm_count) * 4;
    const int grid = grid_for(join ? a.N : (a.N + kRowWarps - 1) / kRowWarps, sm_count * 16);
    auto kern = bits == 8 ? (join ? cache_write_kernel<8, 4, true> : a.D <= 256 ? cache_write_kernel<8, 1, false>
                                  : a.D <= 512 ? cache_write_kernel<8, 2, false> : cache_write_kernel<8, 4, false>)
                          : (join ? cache_write_kernel<4, 4, true> : a.D <= 256 ? cache_write_kernel<4, 1, false>
                                  : a.D <= 512 ? cache_write_kernel<4, 2, false> : cache_write_kernel<4, 4, false>);
    return launch_pdl(kern, dim3(grid), dim3(kRowWarps * 32), 0, stream, a);
}

cudaError_t launch_cache_load(const CacheRowsArgs& a, int bits, int sm_count, cudaStream_t stream) {
    int shift = 0;
    while (shift < 5 && 16 << shift < a.D) ++shift;
    // few wide rows: more lanes a row
    while (shift < 8 && 16 << shift < a.D && (a.N << shift) < static_cast<long long>(sm_count) * 256) ++shift;
    const int wide = a.D % 16 == 0 && a.x_ld % 16 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
    const int grid = grid_for(((a.N << shift) + 255) / 256, sm_count * 8);
    auto kern = bits == 8 ? cache_load_kernel<8> : cache_load_kernel<4>;
    return launch_pdl(kern, dim3(grid), dim3(256), 0, stream, a, shift, wide);
}

}  // namespace attnres
