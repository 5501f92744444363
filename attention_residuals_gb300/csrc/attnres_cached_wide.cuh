// attnres_cached_wide.cuh -- the softmax read over many tokens of compressed
// rows of more than 1024 channels: one warp a token (up to four above 4096
// channels).
//
// A lane owns up to four groups of 32 channels and keeps their FP32 mixture in
// registers, so what a token costs besides its values (the sums over the warp,
// the softmax, addresses) is paid once for up to 4096 channels, and warps wait
// for nobody.  Segments of records come to the warp's own shared memory by
// bulk copies, one a record; per segment
//   1. dots with the query, halves by halves with FP32 sums (fma.rn.f32.f16),
//      a block of rows at a time, so that the query is read once a block; the
//      lanes' sums go to memory, where lane s adds row s's (five shuffles a
//      block, each waiting for the one before, where that room would cost
//      another segment)
//   2. the running softmax, a lane a row
//   3. mixture: codes decoded again, widened and added in FP32; a slot that
//      has been read takes the next segment's record at once.
// What bounds it: instruction issue.  Decoding costs half an instruction a
// value and pass, the dot one, widening one, the packed FMA a half; at eight
// warps an SM (the mixture fills the registers) half of the slots issue.
// S=10 N=32768 D=4096 with the output norm: 294 us in 4 bits (3.4 TB/s), 360
// us in 8 (4.6 TB/s); 8 blocks and a live row, N=16384, R=1024, 8 bits: 140 us
// (5.9 TB/s).  Twelve warps with spills took 383 us for 318, two warps of two
// groups a token 320, a barrier of its own for a segment's first rows 300 for
// 294, slots for a segment ahead (half as long segments) 321 for 299: the
// steps between two segments' rows cost 0.8 us a token.  Dots by shuffles and
// the softmax's sum over the warp once a segment: 299 for 294, S=64 N=8192
// D=8192 in 8 bits 1196 for 1145.
#pragma once

#include <type_traits>

#include "cached_stage.cuh"
#include "kernels.cuh"
#include "launch_pdl.cuh"

namespace attnres {
namespace {

__device__ unsigned g_cached_wide_error;

constexpr int kWideSmem = 227 * 1024;
constexpr uint32_t kDotRow = 36 * 4;  // bytes of a row's 32 dots, a lane each (padded: lanes read four of their own row's at once)

struct WidePlan {
    int seg;                  // records a segment, and slots a warp
    int dots;                 // whether a warp has room for its lanes' dots of a segment
    uint32_t slot;            // bytes of a slot: the warp's part of a record
    uint32_t codes, scales;   // of a slot: bytes of codes, where the scales begin
    uint32_t stat;            // where the statistic is in a slot
    uint32_t q_at, w_at, rows_at, abort_at, warp_at, warp_bytes;  // shared memory: the CTA's, then the warps'
    uint32_t red_at, coef_at, z_at, bar_at, live_at, dots_at;       // in a warp's
    size_t smem;
};

WidePlan wide_plan(int D, int S, bool live, bool norm, int bits, int nc, int w, int warps) {
    WidePlan p{};
    const uint32_t rec = cache_row_bytes(D, bits), codes = cache_code_bytes(D, bits), stat = cache_stat_offset(D, bits);
    const int SL = S + (live ? 1 : 0);
    if (w == 1) {
        p.slot = rec;
        p.codes = p.scales = codes;
        p.stat = stat;
    } else {  // the warp's codes, its scales, and the 16 bytes that hold the statistic
        p.codes = p.scales = static_cast<uint32_t>(nc) * 32 * 4 * bits;
        p.slot = p.codes + nc * 32 + 16;
        p.stat = p.codes + nc * 32 + stat % 16;
    }
    uint32_t off = 0;
    auto take = [&](uint32_t bytes) {
        const uint32_t at = off;
        off += (bytes + 15u) & ~15u;
        return at;
    };
    p.q_at = take(nc * w * 32 * 64);
    p.w_at = take(norm ? nc * w * 32 * 64 : 0);
    p.rows_at = take(S * 8);
    p.abort_at = take(32);  // and the query's factor
    p.warp_at = off;
    off = 0;
    p.bar_at = take(16);  // of the rows and of the live row
    p.live_at = take(live ? nc * 2048 : 0);
    p.z_at = take(2 * SL * 4);
    p.red_at = take(w > 1 ? 2 * 32 * 4 : 0);
    p.coef_at = take(32 * 4);
    // lanes behind a row's last group read on from its end
    const uint32_t lanes = static_cast<uint32_t>(nc) * 32 * 4 * bits, over = lanes > p.slot ? lanes - p.slot : 0;
    const uint32_t room = (kWideSmem - p.warp_at - over) / warps - off - 16;
    int most = static_cast<int>(room / p.slot);
    if (most > 30) most = 30;
    if (most < 1) most = 1;
    const int n = (S + most - 1) / most;
    p.seg = (S + n - 1) / n;
    // not at the price of another segment: S=32 N=16384 D=2048 and a live row,
    // 4 bits, 201 us in four segments without the room, 214 in five with it
    p.dots = p.seg * (p.slot + kDotRow) <= room;
    p.dots_at = off + p.seg * p.slot;
    p.warp_bytes = p.dots_at + p.dots * p.seg * kDotRow;
    p.smem = p.warp_at + static_cast<size_t>(warps) * p.warp_bytes + over;
    return p;
}

// The query's channels c0 .. c0 + 31 as halves times 2^sh, zero outside the
// key.  sh puts the query's largest magnitude in [2^14, 2^15).  bf16 has fewer
// significand bits than a half, so every channel down to 2^-28 of the largest
// is exact; a smaller one is off by at most 2^-39 of the largest.
__device__ __forceinline__ void query_halves(const CachedArgs& a, int c0, int sh, uint32_t (&q)[16]) {
    const float up = __uint_as_float(static_cast<uint32_t>(sh + 127) << 23);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int j = c0 + 2 * i - a.ko;
        const float x = j >= 0 && j < a.R ? bf16_bits_to_float(__ldg(a.q + j)) : 0.0f;
        const float y = j + 1 >= 0 && j + 1 < a.R ? bf16_bits_to_float(__ldg(a.q + j + 1)) : 0.0f;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(q[i]) : "f"(y * up), "f"(x * up));
    }
}

// Maximum over the warp, as integers of the same order.  A NaN counts as above
// or below everything; the weights are NaN then either way.
__device__ __forceinline__ float top_of(float z) {
    const int b = __float_as_int(z), m = __reduce_max_sync(0xffffffffu, b ^ (b >> 31 & 0x7fffffff));
    return __int_as_float(m ^ (m >> 31 & 0x7fffffff));
}

// DOTS: the warp has room for its lanes' dots of a segment.
template <int BITS, int NC, int W, int WARPS, bool NORM, bool LIVE, bool DOTS>
__global__ void __launch_bounds__(32 * WARPS, 1) cached_wide_kernel(const CachedArgs a, const WidePlan pl) {
    constexpr int CH = BITS / 4;                  // 16-byte chunks of codes a group
    constexpr int K = BITS == 8 ? 2 : 4;          // rows of a block of dots
    constexpr int TEAMS = WARPS / W;     // tokens of the CTA at a time
    extern __shared__ __align__(16) unsigned char dyn[];
    const uint32_t sm = smem_u32(dyn);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int team = warp / W, w = warp % W;
    const int SL = a.S + (LIVE ? 1 : 0), seg = pl.seg, nseg = (a.S + seg - 1) / seg;
    const unsigned char** rows = reinterpret_cast<const unsigned char**>(dyn + pl.rows_at);
    volatile int* abort = reinterpret_cast<volatile int*>(dyn + pl.abort_at);
    unsigned char* own = dyn + pl.warp_at + warp * pl.warp_bytes;
    unsigned char* own0 = dyn + pl.warp_at + team * W * pl.warp_bytes;  // of the team's first warp
    const uint32_t bar = smem_u32(own) + pl.bar_at;
    const uint32_t slots = smem_u32(own) + pl.coef_at + 128;
    float* zbuf = reinterpret_cast<float*>(own + pl.z_at);    // logits, then 1 / RMS (of the team's first warp)
    float* coef = reinterpret_cast<float*>(own + pl.coef_at);
    float* dot_rows = reinterpret_cast<float*>(own + pl.dots_at);
    if (threadIdx.x == 0) *abort = 0;
    if (lane == 0) {
        for (int i = 0; i < 2; ++i) mbar_init(reinterpret_cast<uint64_t*>(own + pl.bar_at + 8 * i), 1);
        mbar_fence_init();
    }
    for (int s = threadIdx.x; s < a.S; s += blockDim.x) rows[s] = a.rows[s];
    pdl_wait();

    // 8 bits: a lane's 32 bytes of codes are read as two halves, the second
    // first where that keeps the lanes of a phase on different banks; its
    // channels are then those halves in that order.
    const int sw = BITS == 8 ? (lane >> 2) & 1 : 0;
    uint32_t has = 0, keys = 0, whole = 0;  // bit c: the lane's group c exists, has key channels, has no others
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int c0 = (w * 32 * NC + c * 32 + lane) * 32;
        if (c0 < a.D) has |= 1u << c;
        if (c0 < a.D && c0 < a.ko + a.R && c0 + 32 > a.ko) keys |= 1u << c;
        if (c0 >= a.ko && c0 + 32 <= a.ko + a.R) whole |= 1u << c;
    }
    const uint32_t any_keys = __reduce_or_sync(0xffffffffu, keys), all_whole = __reduce_and_sync(0xffffffffu, whole);
    // channels of register pairs 0-7 and 8-15 of group c
    auto chan = [&](int c, int i) { return (w * 32 * NC + c * 32 + lane) * 32 + 16 * (i ^ sw); };
    {  // the largest magnitude of the query, as bf16 bits
        uint32_t m = 0;
#pragma unroll 8
        for (int j = threadIdx.x; j < a.R; j += blockDim.x) m = max(m, static_cast<uint32_t>(__ldg(a.q + j)) & 0x7fffu);
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) reinterpret_cast<uint32_t*>(own + pl.coef_at)[0] = m;
    }
    __syncthreads();
    uint32_t top = 0;
    for (int i = lane; i < WARPS; i += 32)
        top = max(top, *reinterpret_cast<const uint32_t*>(dyn + pl.warp_at + i * pl.warp_bytes + pl.coef_at));
    const int sh = min(141 - static_cast<int>(__reduce_max_sync(0xffffffffu, top) >> 7), 114);
    const float back = __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
    // the query and the output's weight, in the order of each lane's registers
    for (int e = warp; e < NC * W; e += WARPS) {  // group e * 32 + lane
        uint32_t q[16];
        query_halves(a, (e * 32 + lane) * 32, sh, q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // 8 bits, halves swapped: quad i of the registers is quad i ^ 2 of the channels
            const uint4 x = make_uint4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
            sts128(sm + pl.q_at + ((e * 4 + (i ^ (2 * sw))) * 32 + lane) * 16, x);
            if constexpr (NORM) {
                const int j = (e * 32 + lane) * 32 + 8 * i;
                sts128(sm + pl.w_at + ((e * 4 + (i ^ (2 * sw))) * 32 + lane) * 16,
                       j < a.D ? __ldg(reinterpret_cast<const uint4*>(a.w_o + j)) : make_uint4(0u, 0u, 0u, 0u));
            }
        }
    }
    __syncthreads();  // the last of the CTA's

    // Where the lane's codes and scale of group 0 lie in slot 0.  Lanes behind
    // the row's last group read on, whatever is there, and use nothing of it.
    const uint32_t code0 = slots + lane * (16 * CH) + 16 * sw, code1 = slots + lane * 32 + 16 * (1 - sw);  // (8 bits)
    const uint32_t scale0 = slots + pl.scales + lane;
    // 8 bits: the lane's last group ends in its first half, the second is not codes
    const bool cut = BITS == 8 && a.D % 32 != 0 && a.D % 32 <= 16 &&
                     a.D / 32 >= w * 32 * NC && a.D / 32 < (w + 1) * 32 * NC && a.D / 32 % 32 == lane;
    const int cut_c = a.D / 32 / 32 - w * NC;
    const bool any_cut = BITS == 8 && a.D % 32 != 0 && a.D % 32 <= 16;
    auto codes = [&](uint32_t at, int c) {
        CacheCodes<BITS> x;
        const uint4 u = lds128(code0 + at + c * (512 * CH));
        x.w[0] = u.x, x.w[1] = u.y, x.w[2] = u.z, x.w[3] = u.w;
        if constexpr (CH == 2) {
            const uint4 v = lds128(code1 + at + c * (512 * CH));
            x.w[4] = v.x, x.w[5] = v.y, x.w[6] = v.z, x.w[7] = v.w;
        }
        return x;
    };
    // bytes of this warp's part of a record, and its copy into slot r
    const uint32_t code_bytes = W == 1 ? pl.slot : min(a.codes - w * pl.codes, pl.codes);
    const uint32_t rec = W == 1 ? pl.slot : ((a.stat + 8 + 15) & ~15u);
    const uint32_t scale_bytes = W == 1 ? 0 : min(rec - (a.codes + w * NC * 32), static_cast<uint32_t>(NC) * 32);
    const uint32_t part_bytes = W == 1 ? pl.slot : code_bytes + scale_bytes + 16;
    auto fetch = [&](long long n, int s, int r) {
        const unsigned char* p = rows[s] + n * a.row_ld;
        const uint32_t dst = slots + r * pl.slot;
        bulk_load(dst, p + (W == 1 ? 0 : w * pl.codes), code_bytes, bar);
        if constexpr (W > 1) {
            bulk_load(dst + pl.scales, p + a.codes + w * NC * 32, scale_bytes, bar);
            bulk_load(dst + pl.stat / 16 * 16, p + a.stat / 16 * 16, 16, bar);
        }
    };
    auto expect = [&](int cnt) {
        if (lane == 0) mbar_expect(bar, cnt * part_bytes);
        __syncwarp();
    };
    const uint32_t live_bytes = min((a.D - w * 1024 * NC) * 2u, 2048u * NC);
    auto fetch_live = [&](long long n) {
        if (lane == 0) {
            mbar_expect(bar + 8, live_bytes);
            bulk_load(smem_u32(own) + pl.live_at, a.live + n * a.live_ld + w * 1024 * NC, live_bytes, bar + 8);
        }
    };
    const bool wide = a.D % 16 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 31u) == 0;
    const float inv_D = 1.0f / static_cast<float>(a.D), inv_R = 1.0f / static_cast<float>(a.R);
    int flip = 0;
    // sums over the team's warps of what lane-wise values `x` of each are (buffers in turn)
    auto exchange = [&](float x) {
        if constexpr (W > 1) {
            const unsigned char* r = own0 + pl.red_at + (flip * 32 + lane) * 4;
            *reinterpret_cast<float*>(own + pl.red_at + (flip * 32 + lane) * 4) = x;
            named_bar_sync(team + 1, 32 * W);
            x = *reinterpret_cast<const float*>(r);
#pragma unroll
            for (int u = 1; u < W; ++u) x += *reinterpret_cast<const float*>(r + u * pl.warp_bytes);
            flip ^= 1;
        }
        return x;
    };

    const long long first = static_cast<long long>(blockIdx.x) * TEAMS + team, stride = static_cast<long long>(gridDim.x) * TEAMS;
    uint32_t phases = 0;  // bit i: the parity barrier i is waited for next
    uint32_t stuck = 0, stuck_phases = 0;  // waits that ran out (here or in another warp): nothing more is fetched
    auto wait = [&](int i) {
        if (!mbar_wait_s(bar + 8 * i, phases >> i & 1u, abort, &g_cached_wide_error, kSiteCached) && !(stuck >> i & 1u))
            stuck |= 1u << i, stuck_phases |= (phases >> i & 1u) << i;
        phases ^= 1u << i;
    };
    if (first < a.N) {
        const int cnt = min(seg, a.S);
        expect(cnt);
        if (lane < cnt) fetch(first, lane, lane);
        if constexpr (LIVE) fetch_live(first);
    }
    for (long long n = first; n < a.N; n += stride) {
        f2 acc[NC][16];
        float mx, sum;  // of the softmax: the maximum, and the lane's part of the sum
        if constexpr (LIVE) {  // the live source first: it is the mixture, with weight 1
            float p0 = 0.0f, p1 = 0.0f;
            wait(1);
            const uint32_t x = smem_u32(own) + pl.live_at - w * 2048 * NC;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = chan(c, i / 2) + 8 * (i & 1);
                    const uint4 u = j < a.D ? lds128(x + j * 2) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[c][4 * i + k] = f2_bf16(u4_get(u, k));
                }
            }
            read_done(acc[NC - 1][15]);
            if (n + stride < a.N && !*abort) fetch_live(n + stride);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (!(any_keys >> c & 1u)) continue;
                f2 d = 0ull, s2 = 0ull;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 q = lds128(sm + pl.q_at + (((w * NC + c) * 4 + i) * 32 + lane) * 16);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const f2 v = acc[c][4 * i + k];
                        d = f2_fma(v, f2_half(u4_get(q, k)), d);
                        if (all_whole >> c & 1u) {
                            s2 = f2_fma(v, v, s2);
                        } else {
                            const int j = chan(c, i / 2) + 8 * (i & 1) + 2 * k - a.ko;
                            const float2 y = f2_get(v);
                            s2 = f2_fma(v, f2_make(j >= 0 && j < a.R ? y.x : 0.0f, j + 1 >= 0 && j + 1 < a.R ? y.y : 0.0f), s2);
                        }
                    }
                }
                if (keys >> c & 1u) p0 += f2_sum(d) * back, p1 += f2_sum(s2);
            }
            p0 = warp_sum(p0);
            p1 = warp_sum(p1);
            if constexpr (W > 1) {
                const float both = exchange(lane == 0 ? p0 : p1);
                p0 = __shfl_sync(0xffffffffu, both, 0);
                p1 = __shfl_sync(0xffffffffu, both, 1);
            }
            const float rs = rsqrtf(p1 * inv_R + a.eps);
            mx = a.scale * rs * p0;
            sum = mx != mx ? mx : lane == 0 ? 1.0f : 0.0f;  // a NaN stays one
            if (w == 0 && lane == 0) zbuf[a.S] = mx, zbuf[SL + a.S] = rs;
        } else {
            mx = __uint_as_float(0xff800000u);
            sum = 0.0f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[c][i] = 0ull;
            }
        }
        for (int g = 0; g < nseg; ++g) {
            const int s0 = g * seg, cnt = min(seg, a.S - s0);
            wait(0);
            // what the slots take next
            const bool last = g == nseg - 1;
            const long long nn = last ? n + stride : n;
            const int ns0 = last ? 0 : s0 + seg;
            const int ncnt = nn < a.N && !*abort ? min(seg, a.S - ns0) : 0;
            float dot = 0.0f;  // of row `lane`
            if (any_keys) {
                auto dots = [&](auto count, int r0) {
                    constexpr int M = decltype(count)::value;
                    float p[M];
                    uint32_t at[M];
#pragma unroll
                    for (int r = 0; r < M; ++r) p[r] = 0.0f, at[r] = (r0 + r) * pl.slot;
#pragma unroll 1
                    for (int c = 0; c < NC; ++c) {  // a loop: unrolled, the kernel would not stay in the instruction cache
                        if (!(any_keys >> c & 1u)) continue;
                        const bool key = keys >> c & 1u;
                        uint4 q[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) q[i] = lds128(sm + pl.q_at + (((w * NC + c) * 4 + i) * 32 + lane) * 16);
                        CacheCodes<BITS> x[M];
                        float f[M];
#pragma unroll
                        for (int r = 0; r < M; ++r) x[r] = codes(at[r], c), f[r] = cache_scale(lds8(scale0 + at[r] + c * 32));
                        if (any_cut && cut && c == cut_c) {
#pragma unroll
                            for (int r = 0; r < M; ++r) {
#pragma unroll
                                for (int i = 0; i < BITS; ++i)
                                    if (i / 4 != sw) x[r].w[i] = 0u;
                            }
                        }
#pragma unroll
                        for (int r = 0; r < M; ++r) {
                            uint32_t h[16];
                            x[r].unpack(h);
                            float d0 = 0.0f, d1 = 0.0f;
#pragma unroll
                            for (int i = 0; i < 16; ++i) half2_dot(h[i], u4_get(q[i / 4], i % 4), d0, d1);
                            p[r] += key ? (d0 + d1) * f[r] : 0.0f;
                        }
                    }
                    if constexpr (DOTS) {
#pragma unroll
                        for (int r = 0; r < M; ++r) dot_rows[(r0 + r) * (kDotRow / 4) + lane] = p[r];
                    } else {
                        lanes_sum_to<32>(p, coef + r0);
                    }
                };
                int r = 0;
#pragma unroll 1
                for (; r + K <= cnt; r += K) dots(std::integral_constant<int, K>{}, r);
                if (K == 4 && r + 2 <= cnt) dots(std::integral_constant<int, 2>{}, r), r += 2;
                if (r < cnt) dots(std::integral_constant<int, 1>{}, r);
                __syncwarp();
                if (lane < cnt) {
                    if constexpr (DOTS) {  // lane s adds row s's over the lanes: one wait for a segment, not five shuffles for each block
                        f2 d0 = 0ull, d1 = 0ull;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(dot_rows + lane * (kDotRow / 4) + 4 * i);
                            d0 = f2_add(d0, x.x), d1 = f2_add(d1, x.y);
                        }
                        dot = f2_sum(f2_add(d0, d1));
                    } else {
                        dot = coef[lane];
                    }
                }
            }
            // logits and weights of the segment: lane s has row s
            dot = exchange(dot) * back;
            float z = __uint_as_float(0xff800000u);
            if (lane < cnt) {
                const uint32_t at = slots + lane * pl.slot + pl.stat;
                const bool good = lds32(at + 4) == a.tag;
                if (!good && w == 0) atomicCAS(&g_cached_wide_error, 0u, static_cast<unsigned>(kSiteCacheTag));
                const float rs = good ? rsqrtf(__uint_as_float(lds32(at)) + a.eps) : __uint_as_float(0x7fc00000u);
                z = a.scale * rs * dot;
                if (w == 0) zbuf[s0 + lane] = z, zbuf[SL + s0 + lane] = rs;
            }
            const float mnew = fmaxf(mx, top_of(z));
            const float e = lane < cnt ? __expf(z - mnew) : 0.0f, corr = __expf(mx - mnew);
            __syncwarp();
            coef[lane] = e;
            sum = sum * corr + e;
            mx = mnew;
            if (LIVE || g > 0) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[c][i] = f2_mul(acc[c][i], f2_dup(corr));
                }
            }
            if (ncnt) expect(ncnt);
            else __syncwarp();
            auto mix = [&](int r) {
                const uint32_t at = r * pl.slot;
                const float er = coef[r];
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    uint32_t h[16];
                    codes(at, c).unpack(h);
                    const float f = er * cache_scale(lds8(scale0 + at + c * 32));
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[c][i] = f2_fma(f2_half(h[i]), f2_dup(f), acc[c][i]);
                }
            };
            int r = 0;
#pragma unroll 1
            for (; r + 2 <= cnt; r += 2) {
#pragma unroll 1
                for (int u = 0; u < 2; ++u) mix(r + u);
                read_done(acc[NC - 1][15]);  // both slots are read: they take the next segment's records
                if (lane < 2 && r + lane < ncnt) fetch(nn, ns0 + r + lane, r + lane);
            }
            if (r < cnt) {
                mix(r);
                read_done(acc[NC - 1][15]);
            }
            if (r + lane < ncnt) fetch(nn, ns0 + r + lane, r + lane);
        }
        float post;
        if constexpr (NORM) {
            if (any_cut && cut) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c == cut_c && i / 8 != sw) acc[c][i] = 0ull;
                }
            }
            float s1 = 0.0f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                f2 ss = 0ull;
#pragma unroll
                for (int i = 0; i < 16; ++i) ss = f2_fma(acc[c][i], acc[c][i], ss);
                if (has >> c & 1u) s1 += f2_sum(ss);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {  // both at once
                const float x = __shfl_xor_sync(0xffffffffu, s1, o), y = __shfl_xor_sync(0xffffffffu, sum, o);
                s1 += x, sum += y;
            }
            const float inv = 1.0f / sum;
            s1 = exchange(s1);
            const float o_rstd = rsqrtf(s1 * inv * inv * inv_D + a.eps);
            if (w == 0 && lane == 0) a.o_rstd[n] = o_rstd;
            post = inv * o_rstd;
        } else {
            sum = warp_sum(sum);
            post = 1.0f / sum;
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            uint32_t o[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (NORM) {
                    const uint4 u = lds128(sm + pl.w_at + (((w * NC + c) * 4 + i) * 32 + lane) * 16);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        o[4 * i + k] = f2_to_bf16(f2_mul(f2_mul(acc[c][4 * i + k], f2_dup(post)), f2_bf16(u4_get(u, k))));
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[4 * i + k] = f2_to_bf16(f2_mul(acc[c][4 * i + k], f2_dup(post)));
                }
            }
            const int half[2] = {chan(c, 0), chan(c, 1)};
            store_halves(a.y + n * a.D, half, a.D, wide, o);
        }
        if (w == 0) {
            __syncwarp();
            for (int s = lane; s < SL; s += 32) {
                const float z = zbuf[s];
                a.logit[n * SL + s] = z;
                a.rstd[n * SL + s] = zbuf[SL + s];
                a.alpha[n * SL + s] = __expf(z - mx) / sum;
            }
            __syncwarp();
        }
    }
    if (stuck) {  // leave no copy of this warp's in flight
        const uint64_t t0 = global_timer_ns();
        for (int i = 0; i < 2; ++i)
            while ((stuck >> i & 1u) && !mbar_test_sleep_s(bar + 8 * i, stuck_phases >> i & 1u, 20000u))
                if (global_timer_ns() - t0 > kWaitLimitNs) break;
    }
}

template <int BITS, int NC, int W, int WARPS>
cudaError_t launch_t(const CachedArgs& a, int sm_count, cudaStream_t stream) {
    const WidePlan p = wide_plan(a.D, a.S, a.live != nullptr, a.w_o != nullptr, BITS, NC, W, WARPS);
    auto with = [&](auto norm, auto live, auto dots) {
        constexpr auto kern =
            cached_wide_kernel<BITS, NC, W, WARPS, decltype(norm)::value, decltype(live)::value, decltype(dots)::value>;
        int fit = 0;
        const cudaError_t err = kernel_fit<kern>(32 * WARPS, p.smem, &fit);
        if (err != cudaSuccess) return err;
        const long long teams = WARPS / W, want = (a.N + teams - 1) / teams;
        return launch_pdl(kern, dim3(static_cast<unsigned>(want < sm_count ? want : sm_count)), dim3(32 * WARPS), p.smem,
                          stream, a, p);
    };
    using Yes = std::true_type;
    using No = std::false_type;
    auto run = [&](auto norm, auto live) { return p.dots ? with(norm, live, Yes{}) : with(norm, live, No{}); };
    return a.w_o ? (a.live ? run(Yes{}, Yes{}) : run(Yes{}, No{})) : (a.live ? run(No{}, Yes{}) : run(No{}, No{}));
}

template <int BITS>
cudaError_t launch_bits(const CachedArgs& a, int sm_count, cudaStream_t stream) {
    const int groups = (a.D + 31) / 32;
    // groups a lane, warps a token, warps of an SM (as many as the registers
    // allow without spilling).  Measured while the first of each took so long
    // (slots refilled a segment at a time), output norm: S=10 N=32768 D=4096, 4
    // bits 318 us with <4, 1, 8> against 320 (2, 2, 16) and 351 (2, 2, 12), 8
    // bits 387 against 401 and 432; S=64 N=8192 D=8192, 4 bits 904 with
    // <2, 4, 16> against 956 (4, 2, 8) and 941 (2, 4, 12).
    if (groups <= 64) return launch_t<BITS, 2, 1, 16>(a, sm_count, stream);
    if (groups <= 96) return launch_t<BITS, 3, 1, 12>(a, sm_count, stream);
    if (groups <= 128) return launch_t<BITS, 4, 1, 8>(a, sm_count, stream);
    if (groups <= 192) return launch_t<BITS, 2, 3, 15>(a, sm_count, stream);
    return launch_t<BITS, 2, 4, 16>(a, sm_count, stream);
}

inline unsigned take_error() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_cached_wide_error, sizeof v) != cudaSuccess) return 0xffffffffu;
    if (v) cudaMemcpyToSymbol(g_cached_wide_error, &zero, sizeof zero);
    return v;
}

}  // namespace
}  // namespace attnres
