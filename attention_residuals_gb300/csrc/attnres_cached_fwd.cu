// attnres_cached_fwd.cu -- the softmax read over compressed cache rows.
//
// A team of threads shares a token, one thread per 32 channels (one scale
// group: a thread's codes have one scale).  Rows come in blocks of four: the
// codes are decoded once into half pairs (exact), multiplied with the query
// (also as halves, see load_query) into FP32 sums, the four dots are added
// over the team, and the online softmax (running maximum and sum) takes the
// block into the FP32 mixture while its half pairs are still in registers.
// The key statistic of a cached row is read from its record; the live bf16
// source, read last, gets its own.
#include "cached.cuh"
#include "kernels.cuh"
#include "launch_pdl.cuh"

namespace attnres {
namespace {

__device__ unsigned g_cached_fwd_error;

constexpr int RB = 4;  // rows per block

// The query's 32 channels of this thread as halves, scaled by a power of two
// that puts the largest magnitude in [2^14, 2^15) (`back` undoes it).  bf16
// has fewer significand bits than a half, so every channel down to 2^-28 of
// the thread's largest is exact; a smaller one is off by at most 2^-39 of the
// largest, less than FP32 sums of the products round.  Channels outside the
// key are zero.
__device__ __forceinline__ void load_query(const CachedArgs& a, int c0, uint32_t (&q)[16], float& back, bool& any) {
    uint32_t b[16];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        uint32_t w = 0;
        const int j = c0 + 2 * i;
        if (j >= a.ko && j < a.ko + a.R) w |= __ldg(a.q + j - a.ko);
        if (j + 1 >= a.ko && j + 1 < a.ko + a.R) w |= static_cast<uint32_t>(__ldg(a.q + j + 1 - a.ko)) << 16;
        b[i] = w;
        m = __vmaxu2(m, w & 0x7fff7fffu);
    }
    const int e = static_cast<int>(max(m & 0xffffu, m >> 16) >> 7);  // biased exponent of the largest
    const int sh = min(141 - e, 114);                                // 2^sh: largest to [2^14, 2^15)
    const float up = __uint_as_float(static_cast<uint32_t>(sh + 127) << 23);
    back = __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float2 f = bf2_to_f2(b[i]);
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(q[i]) : "f"(f.y * up), "f"(f.x * up));
    }
    any = c0 < a.ko + a.R && c0 + 32 > a.ko;
}

// Sums over the team: LW lanes of a warp, and all `warps` of the CTA when a
// team is more than one warp.  `red` is one of two buffers used in turn, so
// one barrier per call is enough.
template <int K, int LW, bool MULTI>
__device__ __forceinline__ void team_sum(float (&v)[K], float* red, int warps) {
#pragma unroll
    for (int o = LW / 2; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < K; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
    if constexpr (MULTI) {
        const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < K; ++i) red[w * K + i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < K; ++i) v[i] = 0.0f;
        for (int u = 0; u < warps; ++u) {
#pragma unroll
            for (int i = 0; i < K; ++i) v[i] += red[u * K + i];
        }
    }
}

template <int BITS, int LW, bool MULTI, bool NORM>
__global__ void __launch_bounds__(256) cached_fwd_kernel(const CachedArgs a) {
    __shared__ float red[2][8 * RB];
    extern __shared__ float zbuf_all[];  // [teams][2 * sources]: logits, reciprocal RMS
    pdl_wait();
    const int warps = blockDim.x >> 5;
    const int T = MULTI ? blockDim.x : LW;
    const int teams = MULTI ? 1 : blockDim.x / LW;
    const int team = MULTI ? 0 : threadIdx.x / LW, t = MULTI ? threadIdx.x : threadIdx.x % LW;
    const int c0 = t * 32;
    const int SL = a.S + (a.live ? 1 : 0);
    float* zbuf = zbuf_all + team * 2 * SL;
    uint32_t q[16];
    float back;
    bool key;
    load_query(a, c0, q, back, key);
    const bool has = c0 < a.D;
    int flip = 0;
    const long long stride = static_cast<long long>(gridDim.x) * teams;
    for (long long base = static_cast<long long>(blockIdx.x) * teams; base < a.N; base += stride) {
        const bool valid = base + team < a.N;
        const long long n = valid ? base + team : a.N - 1;
        float2 acc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = make_float2(0.0f, 0.0f);
        float mx = __uint_as_float(0xff800000u), sum = 0.0f;
        for (int s0 = 0; s0 < a.S; s0 += RB) {
            uint32_t h[RB][16];
            float sc[RB], p[RB], rs[RB];
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const int s = min(s0 + r, a.S - 1);
                const unsigned char* row = a.rows[s] + n * a.row_ld;
                CacheCodes<BITS> w;
#pragma unroll
                for (int i = 0; i < BITS; ++i) w.w[i] = 0u;
                sc[r] = 0.0f;
#pragma unroll
                for (int i = 0; i < BITS / 4; ++i) {
                    const uint32_t at = t * (BITS * 4) + i * 16;
                    if (at < a.codes) {
                        const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + at));
                        w.w[4 * i] = u.x, w.w[4 * i + 1] = u.y, w.w[4 * i + 2] = u.z, w.w[4 * i + 3] = u.w;
                    }
                }
                if (has) sc[r] = cache_scale(__ldg(row + a.codes + t));
                const uint2 st = __ldg(reinterpret_cast<const uint2*>(row + a.stat));
                rs[r] = 1.0f / sqrtf(__uint_as_float(st.x) + a.eps);
                if (st.y != a.tag) {
                    if (t == 0 && valid) atomicCAS(&g_cached_fwd_error, 0u, kSiteCacheTag);
                    rs[r] = __uint_as_float(0x7fc00000u);
                }
                w.unpack(h[r]);
                float d0 = 0.0f, d1 = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) half2_dot(h[r][i], q[i], d0, d1);
                p[r] = key ? (d0 + d1) * back * sc[r] : 0.0f;
            }
            team_sum<RB, LW, MULTI>(p, red[flip], warps);
            flip ^= 1;
            float mnew = mx;
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                p[r] = s0 + r < a.S ? a.scale * rs[r] * p[r] : __uint_as_float(0xff800000u);
                mnew = fmaxf(mnew, p[r]);
            }
            const float corr = expf(mx - mnew);
            mx = mnew;
            sum *= corr;
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] = fmul2(acc[i], make_float2(corr, corr));
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                if (s0 + r >= a.S) break;
                if (t == 0) zbuf[2 * (s0 + r)] = p[r], zbuf[2 * (s0 + r) + 1] = rs[r];
                const float e = expf(p[r] - mnew);
                sum += e;
                const float2 ce = make_float2(e * sc[r], e * sc[r]);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] = ffma2(half2_to_f2(h[r][i]), ce, acc[i]);
            }
        }
        if (a.live) {
            const uint16_t* row = a.live + n * a.live_ld + c0;
            float2 x[16];
            float p[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint4 u = make_uint4(0u, 0u, 0u, 0u);
                if (c0 + 8 * i < a.D) u = __ldg(reinterpret_cast<const uint4*>(row) + i);
#pragma unroll
                for (int k = 0; k < 4; ++k) x[4 * i + k] = bf2_to_f2(u4_get(u, k));
            }
            if (key) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int j = c0 + i - a.ko;
                    if (j >= 0 && j < a.R) {
                        const float v = i & 1 ? x[i / 2].y : x[i / 2].x;
                        p[0] += v * bf16_bits_to_float(__ldg(a.q + j));
                        p[1] += v * v;
                    }
                }
            }
            team_sum<2, LW, MULTI>(p, red[flip], warps);
            flip ^= 1;
            const float rs = 1.0f / sqrtf(p[1] / static_cast<float>(a.R) + a.eps);
            const float z = a.scale * rs * p[0];
            const float mnew = fmaxf(mx, z);
            const float corr = expf(mx - mnew), e = expf(z - mnew);
            mx = mnew;
            sum = sum * corr + e;
            if (t == 0) zbuf[2 * a.S] = z, zbuf[2 * a.S + 1] = rs;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[i] = ffma2(x[i], make_float2(e, e), fmul2(acc[i], make_float2(corr, corr)));
        }
        const float inv = 1.0f / sum;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = fmul2(acc[i], make_float2(inv, inv));
        if constexpr (NORM) {
            float ss[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < 16; ++i) ss[0] += acc[i].x * acc[i].x + acc[i].y * acc[i].y;
            team_sum<1, LW, MULTI>(ss, red[flip], warps);
            flip ^= 1;
            const float o_rstd = 1.0f / sqrtf(ss[0] / static_cast<float>(a.D) + a.eps);
            if (t == 0 && valid) a.o_rstd[n] = o_rstd;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int j = c0 + 2 * i;
                if (j < a.D) {
                    acc[i].x *= o_rstd * bf16_bits_to_float(__ldg(a.w_o + j));
                    acc[i].y *= o_rstd * bf16_bits_to_float(__ldg(a.w_o + j + 1));
                }
            }
        }
        if (MULTI) __syncthreads();
        else __syncwarp();
        if (valid) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (c0 + 8 * i < a.D)
                    *reinterpret_cast<uint4*>(a.y + n * a.D + c0 + 8 * i) =
                        make_uint4(pack_f2(acc[4 * i]), pack_f2(acc[4 * i + 1]), pack_f2(acc[4 * i + 2]),
                                   pack_f2(acc[4 * i + 3]));
            }
            for (int s = t; s < SL; s += T) {
                const float z = zbuf[2 * s];
                a.logit[n * SL + s] = z;
                a.rstd[n * SL + s] = zbuf[2 * s + 1];
                a.alpha[n * SL + s] = expf(z - mx) * inv;
            }
        }
        if (MULTI) __syncthreads();
        else __syncwarp();
    }
}

template <int BITS, int LW, bool MULTI>
cudaError_t launch_t(const CachedArgs& a, int sm_count, cudaStream_t stream) {
    const int block = cached_block(a.D), teams = MULTI ? 1 : block / LW;
    const long long want = (a.N + teams - 1) / teams, most = static_cast<long long>(sm_count) * (512 / block);
    const int grid = static_cast<int>(want < most ? want : most);
    const size_t smem = static_cast<size_t>(teams) * 2 * (a.S + 1) * sizeof(float);
    auto kern = a.w_o ? cached_fwd_kernel<BITS, LW, MULTI, true> : cached_fwd_kernel<BITS, LW, MULTI, false>;
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    return launch_pdl(kern, dim3(grid), dim3(block), smem, stream, a);
}

template <int BITS>
cudaError_t launch_bits(const CachedArgs& a, int sm_count, cudaStream_t stream) {
    switch (cached_team(a.D)) {
        case 1: return launch_t<BITS, 1, false>(a, sm_count, stream);
        case 2: return launch_t<BITS, 2, false>(a, sm_count, stream);
        case 4: return launch_t<BITS, 4, false>(a, sm_count, stream);
        case 8: return launch_t<BITS, 8, false>(a, sm_count, stream);
        case 16: return launch_t<BITS, 16, false>(a, sm_count, stream);
        case 32: return launch_t<BITS, 32, false>(a, sm_count, stream);
        default: return launch_t<BITS, 32, true>(a, sm_count, stream);
    }
}

}  // namespace

unsigned take_cached_fwd_error() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_cached_fwd_error, sizeof v) != cudaSuccess) return 0xffffffffu;
    if (v) cudaMemcpyToSymbol(g_cached_fwd_error, &zero, sizeof zero);
    return v;
}

cudaError_t launch_cached_fwd(const CachedArgs& a, int bits, int sm_count, cudaStream_t stream) {
    return bits == 8 ? launch_bits<8>(a, sm_count, stream) : launch_bits<4>(a, sm_count, stream);
}

}  // namespace attnres
