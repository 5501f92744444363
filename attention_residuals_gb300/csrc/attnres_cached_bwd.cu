// attnres_cached_bwd.cu -- gradient of the softmax read over compressed rows.
//
// With the forward's alpha, rstd and logit (a_s, r_s, z_s), v_s the values the
// records stand for and t_s their key slice:
//   do    = dy, or o_rstd * (h - o * o_rstd^2 * <h, o> / D) with h = w_o * dy
//   da_s  = <do, v_s>,  dz_s = a_s * (da_s - sum_u a_u da_u)
//   dv_s  = a_s * do + [key] (scale dz_s r_s q - dz_s z_s r_s^2 / R * t_s)
//   dq    = sum over tokens and sources of scale dz_s r_s t_s
//   dw_o  = sum over tokens of dy * o * o_rstd
// A team of threads shares a token, one thread per 32 channels; three passes
// over its rows form o (with an output norm), the dots da and the gradients.
// Raw rows, dy and the statistics of the next step are copied to the warp's
// shared memory while one is worked on: whole tokens where two of them fit,
// so that a row is read once, else segments of rows per pass, which after the
// first pass come from L2.  dq and dw_o are summed in registers over the CTA's
// tokens; each CTA writes one partial row and the finalize kernel adds the
// rows in a fixed order.
//
// What bounds it: latency at eight warps an SM (the sums and do fill the
// registers), between bursts of gradient stores.  S=10 N=8192 D=4096 with the
// norm: 255 us in 8 bits, 249 us in 4 (1.09 and 0.92 GB: 4.3 and 3.7 TB/s).
// Twelve warps, one buffer refilled row by row and dw_o in shared memory: 297
// us for 259; without the norm at 168 registers in 4 bits, step 542 us for 467.
#include <type_traits>

#include "cached_stage.cuh"
#include "kernels.cuh"
#include "launch_pdl.cuh"

namespace attnres {
namespace {

__device__ unsigned g_cached_bwd_error;

constexpr int kBwdThreads = 256;      // threads of an SM (up to 255 registers each)
constexpr int kSmemSm = 227 * 1024;   // shared memory of an SM that CTAs can have
constexpr int kResidentWarp = 28 << 10;  // a warp's shared memory up to which whole tokens are kept (8 warps of an SM)
constexpr int kStreamWarp = 18 << 10;    // its target where tokens are streamed (12 warps)

// Shared memory of a warp, in this order: two stages of rows, two of the
// tokens' bf16 rows and statistics, the dots unless they are the CTA's, the
// stages' barriers and (teams of whole warps) the output's weight.
template <int BITS, int LW, bool MULTI>
struct Bwd : RowStage<BITS, LW, MULTI> {
    using R = RowStage<BITS, LW, MULTI>;
    static constexpr bool BULK = LW == 32;
    static constexpr int ROW = BULK ? BulkStage<BITS, MULTI>::ROW : R::ROW;
    __host__ __device__ static int rows(int seg) { return BULK ? BulkStage<BITS, MULTI>::bytes(seg) : R::bytes(seg); }
    __host__ __device__ static int stats(int SL) { return ((3 * SL + 1) * R::TW * 4 + 15) & ~15; }
    __host__ __device__ static int token(int SL, bool live) { return R::BF16 * (live ? 2 : 1) + stats(SL); }
    __host__ __device__ static int dots(int SL) { return MULTI ? 0 : (SL * R::TW * 4 + 15) & ~15; }
    __host__ __device__ static int fixed(int SL, bool live) { return 2 * token(SL, live) + dots(SL) + 16 + (BULK ? R::BF16 : 0); }
    __host__ __device__ static int warp(int seg, int SL, bool live) { return 2 * rows(seg) + fixed(SL, live); }
    // of the CTA, behind the warps': dots in two buffers used in turn, <h, o>,
    // the sources' addresses, the abort flag
    __host__ __device__ static int cta(int warps, int S, int SL) {
        return (MULTI ? (2 * warps * (SL + 1) * 4 + 15) & ~15 : 0) + S * 8 + 16;
    }
};

struct BwdPlan {
    int block, seg, fit, grid;
    size_t smem;
};

template <int BITS, int LW, bool MULTI>
BwdPlan plan_t(int S, bool live, long long N, int D, int sm_count) {
    using G = Bwd<BITS, LW, MULTI>;
    const int SL = S + (live ? 1 : 0), fixed = G::fixed(SL, live);
    BwdPlan p{};
    p.seg = S;
    if (G::warp(S, SL, live) > kResidentWarp) {
        int most = (kStreamWarp - fixed) / (2 * G::ROW);
        if (most < 4) most = 4;
        const int n = (S + most - 1) / most;
        p.seg = (S + n - 1) / n;
    }
    p.block = cached_block(D);
    for (;;) {
        const int warps = p.block / 32;
        p.smem = static_cast<size_t>(warps) * G::warp(p.seg, SL, live) + G::cta(warps, S, SL);
        if (MULTI || p.block == 32 || p.smem <= kSmemSm / 2) break;
        p.block /= 2;
    }
    int by_smem = static_cast<int>(kSmemSm / (p.smem + 1024)), by_regs = kBwdThreads / p.block;
    p.fit = by_smem < by_regs ? by_smem : by_regs;
    if (p.fit < 1) p.fit = 1;
    const long long per = MULTI ? 1 : p.block / 32 * G::TW;
    const long long want = (N + per - 1) / per, most = static_cast<long long>(sm_count) * p.fit;
    p.grid = static_cast<int>(want < most ? want : most);
    return p;
}

template <int BITS, int LW, bool MULTI, bool NORM, bool LIVE>
__global__ void __launch_bounds__(kBwdThreads, 1) cached_bwd_kernel(const CachedBwdArgs b) {
    using G = Bwd<BITS, LW, MULTI>;
    constexpr int CH = G::CH, TW = G::TW;
    extern __shared__ __align__(16) unsigned char dyn[];
    const CachedArgs& a = b.c;
    pdl_wait();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int l = lane % LW, tw = lane / LW;
    const int t = MULTI ? threadIdx.x : l, c0 = t * 32;
    const int SL = a.S + (LIVE ? 1 : 0);
    const int seg = b.seg, nseg = (a.S + seg - 1) / seg;
    const bool resident = nseg == 1;
    const int warp_bytes = G::warp(seg, SL, LIVE);
    unsigned char* mine = dyn + wid * warp_bytes;
    const uint32_t st0 = smem_u32(mine);
    const int tok_at = 2 * G::rows(seg), tok_bytes = G::token(SL, LIVE);
    unsigned char* rest = dyn + warps * warp_bytes;
    float* red = MULTI ? reinterpret_cast<float*>(rest)
                       : reinterpret_cast<float*>(mine + tok_at + 2 * tok_bytes) + tw * SL;
    float* ho_red = red + 2 * warps * SL;  // MULTI
    if (MULTI) rest += (2 * warps * (SL + 1) * 4 + 15) & ~15;
    const unsigned char** rows = reinterpret_cast<const unsigned char**>(rest);
    volatile int* abort = reinterpret_cast<volatile int*>(rest + ((a.S * 8 + 15) & ~15));
    const uint32_t bar = st0 + tok_at + 2 * tok_bytes + G::dots(SL);  // of stage 0; 8 bytes on, of stage 1
    for (int s = threadIdx.x; s < a.S; s += blockDim.x) rows[s] = a.rows[s];
    if (threadIdx.x == 0) *abort = 0;
    BulkStage<BITS, MULTI> bulk;
    if constexpr (G::BULK) {
        bulk.init(a, rows, seg);
        for (int i = lane * 16; i < tok_at + 2 * tok_bytes; i += 512) sts128(st0 + i, make_uint4(0u, 0u, 0u, 0u));
        if (lane == 0) {
            mbar_init(reinterpret_cast<uint64_t*>(mine + (bar - st0)), 1);
            mbar_init(reinterpret_cast<uint64_t*>(mine + (bar - st0) + 8), 1);
            mbar_fence_init();
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the zeros before the copies
    }
    const bool has = c0 < a.D, key = has && c0 < a.ko + a.R && c0 + 32 > a.ko;
    const bool warp_key = __any_sync(0xffffffffu, key);
    // Bulk copies leave codes and bf16 rows as they lie in memory.  8 bits: a
    // thread's 32 bytes of codes are read as two halves, the second first where
    // that keeps the lanes of a phase on different banks, and its channels are
    // those halves in that order.
    const int sw = G::BULK && BITS == 8 ? (lane >> 2) & 1 : 0;
    const int half[2] = {c0 + 16 * sw, c0 + 16 * (1 - sw)};  // channels of pairs 0-7 and 8-15
    auto chan = [&](int i) { return half[i / 8] + 2 * (i % 8); };  // of pair i
    f2 q[16], dq[16], dw[16];
    uint32_t mask = 0;  // bits 2i, 2i + 1: the channels of pair i are in the key
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int j = chan(i) - a.ko;
        const bool x = j >= 0 && j < a.R, y = j + 1 >= 0 && j + 1 < a.R;
        q[i] = f2_make(x ? bf16_bits_to_float(__ldg(a.q + j)) : 0.0f, y ? bf16_bits_to_float(__ldg(a.q + j + 1)) : 0.0f);
        mask |= (x ? 1u : 0u) << (2 * i) | (y ? 1u : 0u) << (2 * i + 1);
        dq[i] = dw[i] = 0ull;
    }
    const bool ragged = __any_sync(0xffffffffu, mask != 0xffffffffu);
    __syncthreads();
    uint32_t code_at[CH], scale_at;
    if constexpr (G::BULK) {
#pragma unroll
        for (int i = 0; i < CH; ++i) code_at[i] = lane * (16 * CH) + (CH == 2 ? (i ^ sw) * 16 : 0);
        scale_at = seg * (512 * CH) + lane;
    } else {
        G::places(seg, code_at, scale_at);
    }
    // 8 channels of a token's bf16 row: pairs 4 i ff.
    auto bf16_part = [&](uint32_t at, int i) {
        if constexpr (G::BULK) return lds128(at + lane * 64 + (i ^ (2 * sw)) * 16);
        else return G::bf16_part(at, i);
    };
    auto scale = [&](uint32_t base, int r) {
        if constexpr (G::BULK) return cache_scale(lds8(base + scale_at + r * 32));
        else return G::scale(base, scale_at, r);
    };
    const uint32_t w_at = bar + 16 + lane * 16;  // [4][32] vectors, in the order of each lane's registers
    if constexpr (G::BULK && NORM) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sts128(w_at + i * 512, chan(4 * i) < a.D ? __ldg(reinterpret_cast<const uint4*>(a.w_o + chan(4 * i))) : make_uint4(0u, 0u, 0u, 0u));
        __syncwarp();
    }
    const float inv_D = 1.0f / static_cast<float>(a.D), inv_R = 1.0f / static_cast<float>(a.R);

    const int per = MULTI ? 1 : warps * TW;
    const long long stride = static_cast<long long>(gridDim.x) * per;
    const long long first = static_cast<long long>(blockIdx.x) * per + (MULTI ? 0 : wid * TW);
    uint32_t phases = 0, inflight = 0;  // bit s: parity that stage s waits for next, and whether copies to it are on their way
    // copies of a segment's rows and, with_token, of the token's other rows and statistics
    auto copy = [&](int stage, int tb, long long n0, int g, bool with_token) {
        const uint32_t tok = st0 + tok_at + tb * tok_bytes;
        const int s0 = g * seg, cnt = min(seg, a.S - s0);
        if constexpr (G::BULK) {
            if (!*abort) {
                const uint32_t b0 = bar + 8 * stage, base = st0 + stage * G::rows(seg);
                if (lane == 0)
                    mbar_expect(b0, cnt * bulk.row_bytes() + (with_token ? bulk.bf16_bytes * (LIVE ? 2 : 1) : 0));
                __syncwarp();
                for (int r = lane; r < cnt; r += 32) bulk.copy_row(a, base, n0, s0 + r, r, b0);
                if (with_token && lane == 0) bulk.copy_bf16(b.dy + n0 * a.D, tok, b0);
                if (LIVE && with_token && lane == 1) bulk.copy_bf16(a.live + n0 * a.live_ld, tok + G::BF16, b0);
                inflight |= 1u << stage;
            }
        } else {
            if (with_token) {
                G::copy_bf16(b.dy, a.D, tok, n0, a.N, a.D);
                if constexpr (LIVE) G::copy_bf16(a.live, a.live_ld, tok + G::BF16, n0, a.N, a.D);
            }
            G::copy(a, rows, st0 + stage * G::rows(seg), seg, n0, s0, cnt);
        }
        if (with_token) {
            const uint32_t st = tok + G::BF16 * (LIVE ? 2 : 1);
            for (int i = lane; i < TW * SL; i += 32) {
                const long long from = TW == 1 ? n0 * SL + i : min(n0 + i / SL, a.N - 1) * SL + i % SL;
                cp_async_4s(st + i * 4, a.alpha + from);
                cp_async_4s(st + (TW * SL + i) * 4, a.rstd + from);
                cp_async_4s(st + (2 * TW * SL + i) * 4, a.logit + from);
            }
            if (NORM && lane < TW) cp_async_4s(st + (3 * TW * SL + lane) * 4, a.o_rstd + min(n0 + lane, a.N - 1));
        }
        cp_async_commit();
    };
    constexpr int kFirst = NORM ? 0 : 1;
    int stage = 0, tb = 0, flip = 0;
    if (first < a.N) {
        copy(0, 0, first, 0, true);
    }
    for (long long n0 = first; n0 < a.N; n0 += stride) {
        const bool valid = n0 + tw < a.N;
        const long long n = valid ? n0 + tw : a.N - 1;
        const bool more = n0 + stride < a.N;
        const uint32_t tok = st0 + tok_at + tb * tok_bytes;
        // alpha, then 1 / RMS and logit, which become the coefficients of q and of t
        float* al = reinterpret_cast<float*>(mine + tok_at + tb * tok_bytes + G::BF16 * (LIVE ? 2 : 1)) + tw * SL;
        float* k1 = al + TW * SL;
        float* k2 = k1 + TW * SL;
        f2 g[16];  // do
        auto load_g = [&](uint32_t at) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 u = bf16_part(at, i);
#pragma unroll
                for (int k = 0; k < 4; ++k) g[4 * i + k] = f2_bf16(u4_get(u, k));
            }
        };
        // makes the rows of (pass, segment) ready and starts the copies of what comes next
        auto next = [&](int pass, int seg_i) {
            if (resident && pass != kFirst) return;
            if (!resident && (seg_i < nseg - 1 || pass < 2))
                copy(stage ^ 1, tb, n0, seg_i < nseg - 1 ? seg_i + 1 : 0, false);
            else if (more)
                copy(stage ^ 1, tb ^ 1, n0 + stride, 0, true);
            else
                cp_async_commit();
            if constexpr (G::BULK) {
                if (mbar_wait_s(bar + 8 * stage, phases >> stage & 1u, abort, &g_cached_bwd_error, kSiteCached))
                    phases ^= 1u << stage, inflight &= ~(1u << stage);
            }
            cp_async_wait<1>();
            __syncwarp();
        };
        auto done = [&](int pass, int seg_i) {
            if (G::BULK && pass == 2) read_done(dq[15]);
            else __syncwarp();
            if (!resident || pass == 2) stage ^= 1;
        };
        if constexpr (NORM) {
            f2 o[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = 0ull;
            for (int u = 0; u < nseg; ++u) {
                next(0, u);
                const uint32_t base = st0 + stage * G::rows(seg);
                const int s0 = u * seg, cnt = min(seg, a.S - s0);
                auto mix = [&](auto count, int r0) {
                    constexpr int K = decltype(count)::value;
                    CacheCodes<BITS> w[K];
                    float c[K];
#pragma unroll
                    for (int r = 0; r < K; ++r)
                        w[r] = G::codes(base, code_at, r0 + r), c[r] = al[s0 + r0 + r] * scale(base, r0 + r);
#pragma unroll
                    for (int r = 0; r < K; ++r) {
                        uint32_t h[16];
                        w[r].unpack(h);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = f2_fma(f2_half(h[i]), f2_dup(c[r]), o[i]);
                    }
                };
                int r = 0;
#pragma unroll 1
                for (; r + 2 <= cnt; r += 2) mix(std::integral_constant<int, 2>{}, r);
                if (r < cnt) mix(std::integral_constant<int, 1>{}, r);
                done(0, u);
            }
            if constexpr (LIVE) {
                const float c = al[a.S];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 x = bf16_part(tok + G::BF16, i);
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[4 * i + k] = f2_fma(f2_bf16(u4_get(x, k)), f2_dup(c), o[4 * i + k]);
                }
            }
            load_g(tok);
            const float r = (al - tw * SL)[3 * TW * SL + tw];
            f2 s2 = 0ull;
            if (has) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint4 w;
                    if constexpr (G::BULK) w = lds128(w_at + i * 512);
                    else w = chan(4 * i) < a.D ? __ldg(reinterpret_cast<const uint4*>(a.w_o + chan(4 * i))) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int j = 4 * i + k;
                        if (valid) dw[j] = f2_fma(g[j], f2_mul(o[j], f2_dup(r)), dw[j]);
                        g[j] = f2_mul(g[j], f2_bf16(u4_get(w, k)));
                        s2 = f2_fma(g[j], o[j], s2);
                    }
                }
            }
            float ho = lanes_sum<LW>(f2_sum(s2));
            if constexpr (MULTI) {
                float* out = ho_red + flip * warps;
                if (lane == 0) out[wid] = ho;
                __syncthreads();
                ho = 0.0f;
                for (int u = 0; u < warps; ++u) ho += out[u];
            }
            const float c = -r * r * ho * inv_D;
            if (has) {
#pragma unroll
                for (int i = 0; i < 16; ++i) g[i] = f2_mul(f2_fma(o[i], f2_dup(c), g[i]), f2_dup(r));
            }
        }
        float* out = MULTI ? red + (flip * warps + wid) * SL : red;
        for (int u = 0; u < nseg; ++u) {
            next(1, u);
            if (!NORM && u == 0) load_g(tok);
            const uint32_t base = st0 + stage * G::rows(seg);
            const int s0 = u * seg, cnt = min(seg, a.S - s0);
            auto dots = [&](auto count, int r0) {
                constexpr int K = decltype(count)::value;
                CacheCodes<BITS> w[K];
                float sc[K], p[K];
#pragma unroll
                for (int r = 0; r < K; ++r) w[r] = G::codes(base, code_at, r0 + r), sc[r] = scale(base, r0 + r);
#pragma unroll
                for (int r = 0; r < K; ++r) {
                    uint32_t h[16];
                    w[r].unpack(h);
                    f2 d0 = 0ull, d1 = d0;
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        d0 = f2_fma(f2_half(h[i]), g[i], d0);
                        d1 = f2_fma(f2_half(h[i + 1]), g[i + 1], d1);
                    }
                    p[r] = has ? (f2_sum(d0) + f2_sum(d1)) * sc[r] : 0.0f;
                }
                lanes_sum_to<LW>(p, out + s0 + r0);
            };
            int r = 0;
#pragma unroll 1
            for (; r + 2 <= cnt; r += 2) dots(std::integral_constant<int, 2>{}, r);
            if (r < cnt) dots(std::integral_constant<int, 1>{}, r);
            done(1, u);
        }
        if constexpr (LIVE) {
            f2 d = 0ull;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 x = bf16_part(tok + G::BF16, i);
#pragma unroll
                for (int k = 0; k < 4; ++k) d = f2_fma(f2_bf16(u4_get(x, k)), g[4 * i + k], d);
            }
            float p[1] = {f2_sum(d)};
            lanes_sum_to<LW>(p, out + a.S);
        }
        if constexpr (MULTI) __syncthreads();
        else __syncwarp();
        float mean = 0.0f;  // sum_u a_u da_u
        for (int s = l; s < SL; s += LW) {
            float d = 0.0f;
            if constexpr (MULTI) {
                for (int u = 0; u < warps; ++u) d += red[(flip * warps + u) * SL + s];
            } else {
                d = red[s];
            }
            const float as = al[s], rs = k1[s];
            mean += as * d;
            k2[s] = -k2[s] * rs * rs * inv_R;  // for dz
            k1[s] = a.scale * rs;
            if constexpr (!MULTI) red[s] = d;
        }
        mean = lanes_sum<LW>(mean);
        for (int s = l; s < SL; s += LW) {
            float d = 0.0f;
            if constexpr (MULTI) {
                for (int u = 0; u < warps; ++u) d += red[(flip * warps + u) * SL + s];
            } else {
                d = red[s];
            }
            const float dz = al[s] * (d - mean);
            k1[s] *= dz;
            k2[s] *= dz;
        }
        flip ^= 1;
        __syncwarp();
        const long long to = (n * b.dsrc_ld + c0) * 2;  // of the thread's first channel in a source's gradient
        const bool put = b.want_dsrc && valid;
        const bool put0 = put && half[0] < a.D, put1 = put && half[1] < a.D;
        for (int u = 0; u < nseg; ++u) {
            next(2, u);
            const uint32_t base = st0 + stage * G::rows(seg);
            const int s0 = u * seg, cnt = min(seg, a.S - s0);
            auto store = [&](int s, const uint32_t (&o)[16]) {
                unsigned char* p = reinterpret_cast<unsigned char*>(b.dsrc[s]) + to;
                if (b.wide_src) {
                    store_half(p + 32 * sw, put0, o);
                    store_half(p + 32 * (1 - sw), put1, o + 8);
                } else if (put) {
                    store_halves(reinterpret_cast<uint16_t*>(p) - c0, half, a.D, false, o);
                }
            };
            // one row's gradient and its part of dq; RAGGED: some thread of the warp has channels outside the key
            auto grad = [&](auto ragged_c, int r, uint32_t (&h)[16], float row_scale) {
                constexpr bool RAGGED = decltype(ragged_c)::value;
                const int s = s0 + r;
                const f2 as = f2_dup(al[s]), x1 = f2_dup(k1[s]);
                const float sc = RAGGED && !mask ? 0.0f : row_scale;
                const float y = valid ? k1[s] * sc : 0.0f, z = k2[s] * sc;
                uint32_t o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if constexpr (RAGGED)
                        h[i] &= (mask >> (2 * i) & 1u ? 0xffffu : 0u) | (mask >> (2 * i + 1) & 1u ? 0xffff0000u : 0u);
                    const f2 v = f2_half(h[i]);
                    dq[i] = f2_fma(v, f2_dup(y), dq[i]);
                    o[i] = f2_to_bf16(f2_fma(v, f2_dup(z), f2_fma(q[i], x1, f2_mul(g[i], as))));
                }
                store(s, o);
            };
            // two rows in turn: one is decoded while the other is worked on
            auto grads = [&](auto ragged_c) {
                uint32_t h0[16], h1[16];
                float sc0, sc1 = 0.0f;
                G::codes(base, code_at, 0).unpack(h0);
                sc0 = scale(base, 0);
#pragma unroll 1
                for (int r = 0; r < cnt; r += 2) {
                    const int r1 = min(r + 1, cnt - 1), r2 = min(r + 2, cnt - 1);
                    G::codes(base, code_at, r1).unpack(h1);
                    sc1 = scale(base, r1);
                    grad(ragged_c, r, h0, sc0);
                    if (r + 1 >= cnt) break;
                    G::codes(base, code_at, r2).unpack(h0);
                    sc0 = scale(base, r2);
                    grad(ragged_c, r + 1, h1, sc1);
                }
            };
            if (!warp_key) {
                for (int r = 0; r < cnt; ++r) {
                    const f2 as = f2_dup(al[s0 + r]);
                    uint32_t o[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = f2_to_bf16(f2_mul(g[i], as));
                    store(s0 + r, o);
                }
            } else if (ragged) {
                grads(std::true_type{});
            } else {
                grads(std::false_type{});
            }
            if (LIVE && u == nseg - 1) {
                const float as = al[a.S], x1 = k1[a.S], y1 = valid ? x1 : 0.0f, y2 = k2[a.S];
                uint32_t o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    uint32_t u = u4_get(bf16_part(tok + G::BF16, i / 4), i % 4);
                    if (!(mask >> (2 * i) & 1u)) u &= 0xffff0000u;
                    if (!(mask >> (2 * i + 1) & 1u)) u &= 0x0000ffffu;
                    const f2 v = f2_bf16(u);
                    dq[i] = f2_fma(v, f2_dup(y1), dq[i]);
                    f2 d = f2_mul(g[i], f2_dup(as));
                    d = f2_fma(q[i], f2_dup(x1), d);
                    o[i] = f2_to_bf16(f2_fma(v, f2_dup(y2), d));
                }
                if (b.dlive && valid) store_halves(b.dlive + n * b.dlive_ld, half, a.D, b.wide_live, o);
            }
            done(2, u);
        }
        tb ^= 1;
    }
    cp_async_wait<0>();
    if constexpr (G::BULK) {  // a wait ran out: leave no copy of this warp's in flight
        const uint64_t t0 = global_timer_ns();
        for (int u = 0; u < 2; ++u)
            while ((inflight >> u & 1u) && !mbar_test_sleep_s(bar + 8 * u, phases >> u & 1u, 20000u))
                if (global_timer_ns() - t0 > kWaitLimitNs) break;
    }
    // One partial row per CTA.  Teams of less than the CTA are added in a fixed
    // order: over the warp's teams by shuffles, over the warps in shared memory.
    const int W = a.R + (NORM ? a.D : 0);
    float* part = b.part + static_cast<size_t>(blockIdx.x) * W;
    if constexpr (MULTI) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float2 x = f2_get(dq[i / 2]), y = f2_get(dw[i / 2]);
            const int j = chan(i / 2) + i % 2;
            if (has && (mask >> i & 1u)) part[j - a.ko] = i % 2 ? x.y : x.x;
            if (NORM && j < a.D) part[a.R + j] = i % 2 ? y.y : y.x;
        }
    } else {
        float* sums = reinterpret_cast<float*>(dyn);  // [2][LW][33], over what the warps had
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float2 x2 = f2_get(dq[i / 2]), y2 = f2_get(dw[i / 2]);
            float x = i % 2 ? x2.y : x2.x, y = i % 2 ? y2.y : y2.x;
#pragma unroll
            for (int o = LW; o < 32; o <<= 1) {
                x += __shfl_xor_sync(0xffffffffu, x, o);
                if constexpr (NORM) y += __shfl_xor_sync(0xffffffffu, y, o);
            }
            dq[i / 2] = i % 2 ? f2_make(f2_get(dq[i / 2]).x, x) : f2_make(x, x2.y);
            dw[i / 2] = i % 2 ? f2_make(f2_get(dw[i / 2]).x, y) : f2_make(y, y2.y);
        }
        for (int u = 0; u < warps; ++u) {
            if (wid == u && tw == 0) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float2 x = f2_get(dq[i / 2]), y = f2_get(dw[i / 2]);
                    float* d0 = sums + l * 33 + i;
                    float* d1 = d0 + LW * 33;
                    *d0 = (u ? *d0 : 0.0f) + (i % 2 ? x.y : x.x);
                    if (NORM) *d1 = (u ? *d1 : 0.0f) + (i % 2 ? y.y : y.x);
                }
            }
            __syncthreads();
        }
        if (wid == 0 && tw == 0 && has) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int j = chan(i / 2) + i % 2;
                if (mask >> i & 1u) part[j - a.ko] = sums[l * 33 + i];
                if (NORM && j < a.D) part[a.R + j] = sums[LW * 33 + l * 33 + i];
            }
        }
    }
}

template <int BITS, int LW, bool MULTI>
cudaError_t launch_t(CachedBwdArgs& b, int grid, int sm_count, cudaStream_t stream) {
    const bool live = b.c.live != nullptr, norm = b.c.w_o != nullptr;
    const BwdPlan p = plan_t<BITS, LW, MULTI>(b.c.S, live, b.c.N, b.c.D, sm_count);
    if (p.grid != grid) return cudaErrorInvalidConfiguration;
    b.seg = p.seg;
    auto run = [&](auto with_norm, auto with_live) {
        constexpr auto kern = cached_bwd_kernel<BITS, LW, MULTI, decltype(with_norm)::value, decltype(with_live)::value>;
        int fit = 0;
        const cudaError_t err = kernel_fit<kern>(p.block, p.smem, &fit);
        return err != cudaSuccess ? err : launch_pdl(kern, dim3(grid), dim3(p.block), p.smem, stream, b);
    };
    using Yes = std::true_type;
    using No = std::false_type;
    return norm ? (live ? run(Yes{}, Yes{}) : run(Yes{}, No{})) : (live ? run(No{}, Yes{}) : run(No{}, No{}));
}

// f(integral constants BITS, LW, MULTI) for a row width and format
template <int BITS, typename F>
auto by_team(int D, F f) {
    using B = std::integral_constant<int, BITS>;
    switch (cached_team(D)) {
        case 1: return f(B{}, std::integral_constant<int, 1>{}, std::false_type{});
        case 2: return f(B{}, std::integral_constant<int, 2>{}, std::false_type{});
        case 4: return f(B{}, std::integral_constant<int, 4>{}, std::false_type{});
        case 8: return f(B{}, std::integral_constant<int, 8>{}, std::false_type{});
        case 16: return f(B{}, std::integral_constant<int, 16>{}, std::false_type{});
        case 32: return f(B{}, std::integral_constant<int, 32>{}, std::false_type{});
        default: return f(B{}, std::integral_constant<int, 32>{}, std::true_type{});
    }
}

}  // namespace

unsigned take_cached_bwd_error() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_cached_bwd_error, sizeof v) != cudaSuccess) return 0xffffffffu;
    if (v) cudaMemcpyToSymbol(g_cached_bwd_error, &zero, sizeof zero);
    return v;
}

int cached_bwd_grid(int S, bool live, long long N, int D, int bits, int sm_count) {
    auto f = [&](auto bb, auto lw, auto multi) {
        return plan_t<decltype(bb)::value, decltype(lw)::value, decltype(multi)::value>(S, live, N, D, sm_count).grid;
    };
    return bits == 8 ? by_team<8>(D, f) : by_team<4>(D, f);
}

cudaError_t launch_cached_bwd(CachedBwdArgs& b, int bits, int grid, int sm_count, cudaStream_t stream) {
    auto f = [&](auto bb, auto lw, auto multi) {
        return launch_t<decltype(bb)::value, decltype(lw)::value, decltype(multi)::value>(b, grid, sm_count, stream);
    };
    return bits == 8 ? by_team<8>(b.c.D, f) : by_team<4>(b.c.D, f);
}

}  // namespace attnres
