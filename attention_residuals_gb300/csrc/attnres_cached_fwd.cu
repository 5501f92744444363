// attnres_cached_fwd.cu -- the softmax read over compressed cache rows, and the
// choice between its two kernels (the other one: attnres_cached_wide.cuh).
//
// A team of threads shares a token, one thread per 32 channels (one scale
// group: a thread's codes have one scale).  The token's rows come in segments,
// the next segment being copied to the warp's shared memory while one is read:
//   1. dots: codes decoded to half pairs (exact) times the query's halves, FP32
//      sums (fma.rn.f32.f16), added over the team
//   2. the running softmax (maximum and sum), by the lanes of every warp
//   3. mixture: codes decoded again, widened and added in FP32
// Decoding twice is cheaper than holding a segment's values: they would take
// four times the registers of the codes.  The key statistic of a cached row is
// read from its record; the live bf16 source, read last, gets its own.  What
// bounds it: with few tokens the chain of a segment's copy, dots, exchange and
// softmax (7 us for up to 152 tokens of S=10 D=4096), else instruction issue.
#include <cstdlib>
#include <type_traits>

#include "cached_stage.cuh"
#include "kernels.cuh"
#include "launch_pdl.cuh"

namespace attnres {
namespace {

__device__ unsigned g_cached_fwd_error;

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
        const float2 f = f2_get(f2_bf16(b[i]));
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(q[i]) : "f"(f.y * up), "f"(f.x * up));
    }
    any = c0 < a.ko + a.R && c0 + 32 > a.ko;
}

constexpr int kStages = 2;
constexpr int kSegmentBytes = 5632;  // of a warp's rows in one stage (20 warps of an SM, two stages: 220 KB)

// Shared memory of a warp: two stages of a segment of rows, the segment's
// coefficients and (unless they are the CTA's) its dots.
template <int BITS, int LW, bool MULTI>
struct Seg : RowStage<BITS, LW, MULTI> {
    using R = RowStage<BITS, LW, MULTI>;
    static constexpr int MOST = kSegmentBytes / R::ROW;
    __host__ __device__ static int rows(int S) {  // rows a segment
        const int n = (S + MOST - 1) / MOST;
        return (S + n - 1) / n;
    }
    __host__ __device__ static int coef(int seg) { return (R::TW * (seg + 2) * 4 + 15) & ~15; }
    __host__ __device__ static int warp(int seg) { return kStages * R::bytes(seg) + 2 * coef(seg); }
};

template <int BITS, int LW, bool MULTI, bool NORM, bool LIVE>
__global__ void __launch_bounds__(256, 2) cached_fwd_kernel(const CachedArgs a) {
    using G = Seg<BITS, LW, MULTI>;
    constexpr int CH = G::CH, TW = G::TW;
    extern __shared__ __align__(16) unsigned char dyn[];
    pdl_wait();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int l = lane % LW, tw = lane / LW;                   // lane of the team, team of the warp
    const int t = MULTI ? threadIdx.x : l;                     // thread of the team
    const int c0 = t * 32;
    const int SL = a.S + (LIVE ? 1 : 0);
    const int seg = G::rows(a.S), nseg = (a.S + seg - 1) / seg;
    unsigned char* mine = dyn + wid * G::warp(seg);
    float* coef = reinterpret_cast<float*>(mine + kStages * G::bytes(seg)) + tw * (seg + 2);
    // dots of a segment: per warp, or for all warps of a team in two buffers used in turn
    unsigned char* rest = dyn + warps * G::warp(seg);
    float* red = MULTI ? reinterpret_cast<float*>(rest)
                       : reinterpret_cast<float*>(mine + kStages * G::bytes(seg) + G::coef(seg)) + tw * (seg + 2);
    if (MULTI) rest += (2 * warps * (seg + 2) * 4 + 15) & ~15;
    float* zbuf = reinterpret_cast<float*>(rest) + (MULTI ? 0 : (wid * TW + tw) * 2 * SL);  // logits, then 1 / RMS
    const unsigned char** rows = reinterpret_cast<const unsigned char**>(
        rest + ((static_cast<size_t>(MULTI ? 1 : warps * TW) * 2 * SL * 4 + 15) & ~size_t(15)));
    for (int s = threadIdx.x; s < a.S; s += blockDim.x) rows[s] = a.rows[s];
    uint32_t q[16];
    float back;
    bool key;
    load_query(a, c0, q, back, key);
    const bool has = c0 < a.D;
    const bool warp_key = __any_sync(0xffffffffu, key);
    const bool wide = a.D % 16 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 31u) == 0;
    __syncthreads();

    // tokens of a CTA step: one for a team of several warps, else TW a warp
    const int per = MULTI ? 1 : warps * TW;
    const long long stride = static_cast<long long>(gridDim.x) * per;
    const long long first = static_cast<long long>(blockIdx.x) * per + (MULTI ? 0 : wid * TW);
    if (first >= a.N) return;  // whole warps only (a team of several warps shares `first`)

    const uint32_t st0 = smem_u32(mine);
    auto issue = [&](int stage, long long n0, int g) {
        G::copy(a, rows, st0 + stage * G::bytes(seg), seg, n0, g * seg, min(seg, a.S - g * seg));
        cp_async_commit();
    };
    uint32_t code_at[CH], scale_at;
    G::places(seg, code_at, scale_at);
    // dots of rows r0 .. r0 + K - 1 with the query, summed over the team's lanes of this warp
    auto dots = [&](auto count, uint32_t base, int r0, float* out) {
        constexpr int K = decltype(count)::value;
        float p[K];
        CacheCodes<BITS> w[K];
        float sc[K];
#pragma unroll
        for (int r = 0; r < K; ++r) w[r] = G::codes(base, code_at, r0 + r), sc[r] = G::scale(base, scale_at, r0 + r);
#pragma unroll
        for (int r = 0; r < K; ++r) {
            uint32_t h[16];
            w[r].unpack(h);
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                half2_dot(h[i], q[i], d[0], d[1]);
                half2_dot(h[i + 1], q[i + 1], d[2], d[3]);
            }
            p[r] = key ? ((d[0] + d[1]) + (d[2] + d[3])) * back * sc[r] : 0.0f;
        }
        lanes_sum_to<LW>(p, out + r0);
    };

    issue(0, first, 0);
    int stage = 0, flip = 0;
    for (long long n0 = first; n0 < a.N; n0 += stride) {
        const bool valid = n0 + tw < a.N;
        const long long n = valid ? n0 + tw : a.N - 1;
        uint4 lv[4];
        if constexpr (LIVE) {
            const uint16_t* x = a.live + n * a.live_ld + c0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                lv[i] = c0 + 8 * i < a.D ? ld_global_nc_v4(x + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
        }
        f2 acc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0ull;
        float mx = __uint_as_float(0xff800000u), sum = 0.0f;
        for (int g = 0; g < nseg; ++g) {
            // the next segment (of this token or the next one) is copied while this one is read
            const bool last = g == nseg - 1;
            if (!last || n0 + stride < a.N) {
                issue(stage ^ 1, last ? n0 + stride : n0, last ? 0 : g + 1);
                cp_async_wait<1>();
            } else {
                cp_async_wait<0>();
            }
            __syncwarp();
            const uint32_t base = st0 + stage * G::bytes(seg);
            const int s0 = g * seg, cnt = min(seg, a.S - s0);
            const bool with_live = LIVE && last;
            float* out = MULTI ? red + (flip * warps + wid) * (seg + 2) : red;
            if (warp_key) {
                int r = 0;
                for (; r + 4 <= cnt; r += 4) dots(std::integral_constant<int, 4>{}, base, r, out);
                if (cnt & 2) dots(std::integral_constant<int, 2>{}, base, r, out), r += 2;
                if (cnt & 1) dots(std::integral_constant<int, 1>{}, base, r, out);
            } else {
                for (int r = l; r < cnt; r += LW) out[r] = 0.0f;
            }
            if (with_live) {
                float p[2] = {0.0f, 0.0f};
                if (key) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int j = c0 + i - a.ko;
                        if (j >= 0 && j < a.R) {
                            const uint32_t w = u4_get(lv[i / 8], i / 2 % 4);
                            const float v = __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
                            p[0] += v * bf16_bits_to_float(__ldg(a.q + j));
                            p[1] += v * v;
                        }
                    }
                }
                lanes_sum_to<LW>(p, out + cnt);
            }
            if constexpr (MULTI) __syncthreads();
            else __syncwarp();
            // logits and weights of the segment, by the lanes of each warp
            float top = __uint_as_float(0xff800000u);
            const int all = cnt + (with_live ? 1 : 0);
            for (int s = l; s < all; s += LW) {
                float dot = 0.0f, ms = 0.0f;
                if constexpr (MULTI) {
                    const float* in = red + flip * warps * (seg + 2) + s;
                    for (int u = 0; u < warps; ++u) dot += in[u * (seg + 2)];
                    if (with_live && s == cnt)
                        for (int u = 0; u < warps; ++u) ms += in[u * (seg + 2) + 1];
                } else {
                    dot = red[s];
                    if (with_live && s == cnt) ms = red[s + 1];
                }
                float rs;
                if (with_live && s == cnt) {
                    rs = rsqrtf(ms / static_cast<float>(a.R) + a.eps);
                } else {
                    const uint2 stv = G::stat(base, seg, s, tw);
                    rs = rsqrtf(__uint_as_float(stv.x) + a.eps);
                    if (stv.y != a.tag) {
                        if (valid) atomicCAS(&g_cached_fwd_error, 0u, static_cast<unsigned>(kSiteCacheTag));
                        rs = __uint_as_float(0x7fc00000u);
                    }
                }
                const float z = a.scale * rs * dot;
                coef[s] = z;
                if (!MULTI || wid == 0) zbuf[s0 + s] = z, zbuf[SL + s0 + s] = rs;
                top = fmaxf(top, z);
            }
            const float mnew = fmaxf(mx, lanes_max<LW>(top));
            float part = 0.0f;
            for (int s = l; s < all; s += LW) {
                const float e = expf(coef[s] - mnew);
                coef[s] = e;
                part += e;
            }
            const float corr = expf(mx - mnew);
            sum = sum * corr + lanes_sum<LW>(part);
            mx = mnew;
            __syncwarp();
            if (g > 0) {
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] = f2_mul(acc[i], f2_dup(corr));
            }
            auto mix = [&](auto count, int r0) {
                constexpr int K = decltype(count)::value;
                CacheCodes<BITS> w[K];
                float c[K];
#pragma unroll
                for (int r = 0; r < K; ++r) w[r] = G::codes(base, code_at, r0 + r), c[r] = coef[r0 + r] * G::scale(base, scale_at, r0 + r);
#pragma unroll
                for (int r = 0; r < K; ++r) {
                    uint32_t h[16];
                    w[r].unpack(h);
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[i] = f2_fma(f2_half(h[i]), f2_dup(c[r]), acc[i]);
                }
            };
            {
                int r = 0;
                for (; r + 4 <= cnt; r += 4) mix(std::integral_constant<int, 4>{}, r);
                if (cnt & 2) mix(std::integral_constant<int, 2>{}, r), r += 2;
                if (cnt & 1) mix(std::integral_constant<int, 1>{}, r);
            }
            if (with_live) {
                const float c = coef[cnt];
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] = f2_fma(f2_bf16(u4_get(lv[i / 4], i % 4)), f2_dup(c), acc[i]);
            }
            __syncwarp();  // the stage and the coefficients are free again
            stage ^= 1;
            flip ^= 1;
        }
        const float inv = 1.0f / sum;
        f2 out2 = f2_dup(inv);
        if constexpr (NORM) {
            f2 ss = 0ull;
#pragma unroll
            for (int i = 0; i < 16; ++i) ss = f2_fma(acc[i], acc[i], ss);
            float s1 = lanes_sum<LW>(has ? f2_sum(ss) : 0.0f);
            if constexpr (MULTI) {
                float* out = red + flip * warps * (seg + 2);
                if (lane == 0) out[wid] = s1;
                __syncthreads();
                s1 = 0.0f;
                for (int u = 0; u < warps; ++u) s1 += out[u];
                flip ^= 1;
            }
            const float o_rstd = rsqrtf(s1 * inv * inv / static_cast<float>(a.D) + a.eps);
            if (t == 0 && valid) a.o_rstd[n] = o_rstd;
            out2 = f2_dup(inv * o_rstd);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (NORM) {
                const uint4 w = c0 + 8 * i < a.D ? __ldg(reinterpret_cast<const uint4*>(a.w_o + c0) + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[4 * i + k] = f2_mul(f2_mul(acc[4 * i + k], out2), f2_bf16(u4_get(w, k)));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[4 * i + k] = f2_mul(acc[4 * i + k], out2);
            }
        }
        if (valid) {
            uint32_t o[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = f2_to_bf16(acc[i]);
            store_bf16x32(a.y + n * a.D + c0, a.D - c0, wide, o);
            if (!MULTI || wid == 0) {
                for (int s = l; s < SL; s += LW) {
                    const float z = zbuf[s];
                    a.logit[n * SL + s] = z;
                    a.rstd[n * SL + s] = zbuf[SL + s];
                    a.alpha[n * SL + s] = expf(z - mx) * inv;
                }
            }
        }
        __syncwarp();
    }
}

// Whether many tokens of wide rows go to the kernel with one to four warps a
// token: it spends fewer instructions a token, but fills the card and pays its
// set-up only over a few tokens a warp.  Measured (us, this kernel against
// that one, S=10 but where noted, output norm, 8 bits / 4 bits):
//   D=1024 (S=8)  N=7296   27 / 21 against 26 / 23: this one at any length
//   D=2048        N=2432   24 / 19 against 18 / 16, N=1216 15 / 12 against 18 / 15
//   D=4096        N=2432   44 / 31 against 43 / 29, N=608 16 / 13 against 20 / 18
//   D=5120        N=7296  146 / 110 against 142 / 114
//   D=8192 (S=64) N=1216  231 / 155 against 185 / 144, N=304 62 / 43 against 99 / 75
bool many_tokens(int D, long long N) { return D > 1024 && N >= (D <= 4096 ? 2400 : D <= 6144 ? 8000 : 1200); }

template <int BITS, int LW, bool MULTI>
cudaError_t launch_t(const CachedArgs& a, int sm_count, cudaStream_t stream) {
    using G = Seg<BITS, LW, MULTI>;
    const int block = cached_block(a.D), warps = block / 32, SL = a.S + (a.live ? 1 : 0);
    const int seg = G::rows(a.S), per = MULTI ? 1 : warps * G::TW;
    size_t smem = static_cast<size_t>(warps) * G::warp(seg);
    if (MULTI) smem += (2 * warps * (seg + 2) * 4 + 15) & ~15;
    smem += (static_cast<size_t>(per) * 2 * SL * 4 + 15) & ~size_t(15);
    smem += static_cast<size_t>(a.S) * 8;
    auto run = [&](auto norm, auto live) {
        constexpr auto kern = cached_fwd_kernel<BITS, LW, MULTI, decltype(norm)::value, decltype(live)::value>;
        int fit = 0;
        const cudaError_t err = kernel_fit<kern>(block, smem, &fit);
        if (err != cudaSuccess) return err;
        const long long want = (a.N + per - 1) / per, most = static_cast<long long>(sm_count) * fit;
        return launch_pdl(kern, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(block), smem, stream, a);
    };
    using Yes = std::true_type;
    using No = std::false_type;
    return a.w_o ? (a.live ? run(Yes{}, Yes{}) : run(Yes{}, No{})) : (a.live ? run(No{}, Yes{}) : run(No{}, No{}));
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
    const char* form = std::getenv("ATTNRES_CACHED_FWD");  // "warp" or "cta": one form wherever it fits (tests)
    const bool warp = form && form[0] == 'w' ? a.D > 1024 : form && form[0] == 'c' ? false : many_tokens(a.D, a.N);
    if (warp)
        return bits == 8 ? launch_cached_wide8(a, sm_count, stream) : launch_cached_wide4(a, sm_count, stream);
    return bits == 8 ? launch_bits<8>(a, sm_count, stream) : launch_bits<4>(a, sm_count, stream);
}

}  // namespace attnres
