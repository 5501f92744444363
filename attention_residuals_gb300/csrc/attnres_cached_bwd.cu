// attnres_cached_bwd.cu -- gradient of the softmax read over compressed rows.
//
// With the forward's alpha, rstd and logit (a_s, r_s, z_s), v_s the values the
// records stand for and t_s their key slice:
//   do    = dy, or o_rstd * (h - o * o_rstd^2 * <h, o> / D) with h = w_o * dy
//   da_s  = <do, v_s>,  dz_s = a_s * (da_s - sum_u a_u da_u)
//   dv_s  = a_s * do + [key] (scale dz_s r_s q - dz_s z_s r_s^2 / R * t_s)
//   dq    = sum over tokens and sources of scale dz_s r_s t_s
//   dw_o  = sum over tokens of dy * o * o_rstd
// A team of threads shares a token, one thread per 32 channels.  The rows are
// read once per pass (the mixture o when there is an output norm, the dots,
// the gradients); after the first they come from L2.  dq and dw_o are FP32
// sums in registers over the CTA's tokens, one partial row per CTA, added in
// a fixed order by the finalize kernel.
#include "cached.cuh"
#include "kernels.cuh"
#include "launch_pdl.cuh"

namespace attnres {
namespace {

__device__ unsigned g_cached_bwd_error;

constexpr int RB = 4;

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

// One row's 32 channels of this thread: half pairs and their scale.
template <int BITS>
__device__ __forceinline__ float load_row(const CachedArgs& a, int s, long long n, int t, bool has, uint32_t (&h)[16]) {
    const unsigned char* row = a.rows[s] + n * a.row_ld;
    CacheCodes<BITS> w;
#pragma unroll
    for (int i = 0; i < BITS; ++i) w.w[i] = 0u;
#pragma unroll
    for (int i = 0; i < BITS / 4; ++i) {
        const uint32_t at = t * (BITS * 4) + i * 16;
        if (at < a.codes) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + at));
            w.w[4 * i] = u.x, w.w[4 * i + 1] = u.y, w.w[4 * i + 2] = u.z, w.w[4 * i + 3] = u.w;
        }
    }
    w.unpack(h);
    return has ? cache_scale(__ldg(row + a.codes + t)) : 0.0f;
}

__device__ __forceinline__ void load_bf16(const uint16_t* p, int c0, int D, float2 (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (c0 + 8 * i < D) u = __ldg(reinterpret_cast<const uint4*>(p + c0) + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[4 * i + k] = bf2_to_f2(u4_get(u, k));
    }
}

__device__ __forceinline__ void store_bf16(uint16_t* p, int c0, int D, const float2 (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (c0 + 8 * i < D)
            *reinterpret_cast<uint4*>(p + c0 + 8 * i) = make_uint4(pack_f2(x[4 * i]), pack_f2(x[4 * i + 1]),
                                                                   pack_f2(x[4 * i + 2]), pack_f2(x[4 * i + 3]));
    }
}

template <int BITS, int LW, bool MULTI, bool NORM>
__global__ void __launch_bounds__(256) cached_bwd_kernel(const CachedBwdArgs b) {
    __shared__ float red[2][8 * RB];
    extern __shared__ float dyn[];
    const CachedArgs& a = b.c;
    pdl_wait();
    const int warps = blockDim.x >> 5;
    const int T = MULTI ? blockDim.x : LW;
    const int teams = MULTI ? 1 : blockDim.x / LW;
    const int team = MULTI ? 0 : threadIdx.x / LW, t = MULTI ? threadIdx.x : threadIdx.x % LW;
    const int c0 = t * 32;
    const int SL = a.S + (a.live ? 1 : 0);
    float* da = dyn + team * SL;  // the token's <do, v_s>
    const bool has = c0 < a.D, key = has && c0 < a.ko + a.R && c0 + 32 > a.ko;
    float2 q[16], dq[16], dw[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int j = c0 + 2 * i - a.ko;
        q[i].x = j >= 0 && j < a.R ? bf16_bits_to_float(__ldg(a.q + j)) : 0.0f;
        q[i].y = j + 1 >= 0 && j + 1 < a.R ? bf16_bits_to_float(__ldg(a.q + j + 1)) : 0.0f;
        dq[i] = dw[i] = make_float2(0.0f, 0.0f);
    }
    // bit i: channel c0 + i is a key channel
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (c0 + i >= a.ko && c0 + i < a.ko + a.R) mask |= 1u << i;
    int flip = 0;
    const long long stride = static_cast<long long>(gridDim.x) * teams;
    for (long long base = static_cast<long long>(blockIdx.x) * teams; base < a.N; base += stride) {
        const bool valid = base + team < a.N;
        const long long n = valid ? base + team : a.N - 1;
        const float* al = a.alpha + n * SL;
        const float* rs = a.rstd + n * SL;
        const float* lg = a.logit + n * SL;
        float2 g[16];  // do
        load_bf16(b.dy + n * a.D, c0, a.D, g);
        if constexpr (NORM) {
            float2 o[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = make_float2(0.0f, 0.0f);
            for (int s = 0; s < a.S; ++s) {
                uint32_t h[16];
                const float sc = load_row<BITS>(a, s, n, t, has, h) * al[s];
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = ffma2(half2_to_f2(h[i]), make_float2(sc, sc), o[i]);
            }
            if (a.live) {
                float2 x[16];
                load_bf16(a.live + n * a.live_ld, c0, a.D, x);
                const float al_s = al[a.S];
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = ffma2(x[i], make_float2(al_s, al_s), o[i]);
            }
            const float r = a.o_rstd[n];
            float2 w[16];
            load_bf16(a.w_o, c0, a.D, w);
            float ho[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (valid) dw[i] = ffma2(g[i], fmul2(o[i], make_float2(r, r)), dw[i]);
                g[i] = fmul2(g[i], w[i]);
                ho[0] += g[i].x * o[i].x + g[i].y * o[i].y;
            }
            team_sum<1, LW, MULTI>(ho, red[flip], warps);
            flip ^= 1;
            const float c = -r * r * ho[0] / static_cast<float>(a.D);
#pragma unroll
            for (int i = 0; i < 16; ++i) g[i] = fmul2(ffma2(o[i], make_float2(c, c), g[i]), make_float2(r, r));
        }
        for (int s0 = 0; s0 < SL; s0 += RB) {
            float p[RB];
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const int s = s0 + r;
                p[r] = 0.0f;
                if (s < a.S) {
                    uint32_t h[16];
                    const float sc = load_row<BITS>(a, s, n, t, has, h);
                    float2 d = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int i = 0; i < 16; ++i) d = ffma2(half2_to_f2(h[i]), g[i], d);
                    if (has) p[r] = (d.x + d.y) * sc;
                } else if (s == a.S && a.live) {
                    float2 x[16];
                    load_bf16(a.live + n * a.live_ld, c0, a.D, x);
                    float2 d = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int i = 0; i < 16; ++i) d = ffma2(x[i], g[i], d);
                    p[r] = d.x + d.y;
                }
            }
            team_sum<RB, LW, MULTI>(p, red[flip], warps);
            flip ^= 1;
            if (t == 0) {
#pragma unroll
                for (int r = 0; r < RB; ++r)
                    if (s0 + r < SL) da[s0 + r] = p[r];
            }
        }
        if (MULTI) __syncthreads();
        else __syncwarp();
        float mean = 0.0f;  // sum_u a_u da_u
        for (int s = 0; s < SL; ++s) mean += al[s] * da[s];
        for (int s = 0; s < SL; ++s) {
            const float as = al[s];
            const float dz = as * (da[s] - mean);
            const float k1 = a.scale * dz * rs[s], k2 = -dz * lg[s] * rs[s] * rs[s] / static_cast<float>(a.R);
            const bool is_live = s == a.S;
            uint16_t* out = is_live ? b.dlive : (b.want_dsrc ? b.dsrc[s] : nullptr);
            const long long ld = is_live ? b.dlive_ld : b.dsrc_ld;
            float2 d[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) d[i] = fmul2(g[i], make_float2(as, as));
            if (key) {
                float2 x[16];
                if (is_live) {
                    load_bf16(a.live + n * a.live_ld, c0, a.D, x);
                } else {
                    uint32_t h[16];
                    const float sc = load_row<BITS>(a, s, n, t, has, h);
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = fmul2(half2_to_f2(h[i]), make_float2(sc, sc));
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (!(mask >> (2 * i) & 1u)) x[i].x = 0.0f;
                    if (!(mask >> (2 * i + 1) & 1u)) x[i].y = 0.0f;
                    d[i] = ffma2(q[i], make_float2(k1, k1), ffma2(x[i], make_float2(k2, k2), d[i]));
                    if (valid) dq[i] = ffma2(x[i], make_float2(k1, k1), dq[i]);
                }
            }
            if (out && valid) store_bf16(out + n * ld, c0, a.D, d);
        }
        if (MULTI) __syncthreads();
        else __syncwarp();
    }
    // one partial row per CTA: the teams' sums are added in team order
    const int W = a.R + (NORM ? a.D : 0);
    float* part = b.part + static_cast<size_t>(blockIdx.x) * W;
    for (int u = 0; u < teams; ++u) {
        if (team == u && has) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float x = i & 1 ? dq[i / 2].y : dq[i / 2].x;
                const float y = i & 1 ? dw[i / 2].y : dw[i / 2].x;
                const int j = c0 + i - a.ko;
                if (mask >> i & 1u) part[j] = u ? part[j] + x : x;
                if (NORM && c0 + i < a.D) part[a.R + c0 + i] = u ? part[a.R + c0 + i] + y : y;
            }
        }
        __syncthreads();
    }
}

template <int BITS, int LW, bool MULTI>
cudaError_t launch_t(const CachedBwdArgs& b, int grid, cudaStream_t stream) {
    const int block = cached_block(b.c.D), teams = MULTI ? 1 : block / LW;
    const size_t smem = static_cast<size_t>(teams) * (b.c.S + 1) * sizeof(float);
    auto kern = b.c.w_o ? cached_bwd_kernel<BITS, LW, MULTI, true> : cached_bwd_kernel<BITS, LW, MULTI, false>;
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    return launch_pdl(kern, dim3(grid), dim3(block), smem, stream, b);
}

template <int BITS>
cudaError_t launch_bits(const CachedBwdArgs& b, int grid, cudaStream_t stream) {
    switch (cached_team(b.c.D)) {
        case 1: return launch_t<BITS, 1, false>(b, grid, stream);
        case 2: return launch_t<BITS, 2, false>(b, grid, stream);
        case 4: return launch_t<BITS, 4, false>(b, grid, stream);
        case 8: return launch_t<BITS, 8, false>(b, grid, stream);
        case 16: return launch_t<BITS, 16, false>(b, grid, stream);
        case 32: return launch_t<BITS, 32, false>(b, grid, stream);
        default: return launch_t<BITS, 32, true>(b, grid, stream);
    }
}

}  // namespace

unsigned take_cached_bwd_error() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_cached_bwd_error, sizeof v) != cudaSuccess) return 0xffffffffu;
    if (v) cudaMemcpyToSymbol(g_cached_bwd_error, &zero, sizeof zero);
    return v;
}

int cached_bwd_grid(long long N, int D, int sm_count) {
    const int block = cached_block(D), team = cached_team(D), teams = team > 32 ? 1 : block / team;
    const long long want = (N + teams - 1) / teams, most = static_cast<long long>(sm_count) * (512 / block);
    return static_cast<int>(want < most ? want : most);
}

cudaError_t launch_cached_bwd(const CachedBwdArgs& b, int bits, int grid, cudaStream_t stream) {
    return bits == 8 ? launch_bits<8>(b, grid, stream) : launch_bits<4>(b, grid, stream);
}

}  // namespace attnres
