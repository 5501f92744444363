// cached_stage.cuh -- raw cache rows in a warp's own part of shared memory
// (the read over cached rows and its gradient).
//
// A team of threads shares a token, one thread per 32 channels: LW lanes of a
// warp, or the whole CTA (MULTI) when a row has more than 1024 channels.  A
// warp copies the codes of its 32 threads, their scales and the statistics of
// its tokens by itself and waits for them by itself, so the copies need no
// barrier wider than the warp.
#pragma once

#include "cached.cuh"

namespace attnres {

// 16-byte asynchronous copy past L1; zeros where !on (the source is not read).
__device__ __forceinline__ void cp_async_16z(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_8s(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_4s(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// Announce `bytes` to the barrier at shared address `bar` (one arrival).
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

// All lanes meet here, each after `v`, which must be computed from the last
// shared-memory loads of what is then overwritten by a bulk copy: the vote
// cannot issue while a load is in flight.
__device__ __forceinline__ void read_done(f2 v) {
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.eq.u64 p, %0, 0x7fc12345;\n\tvote.sync.any.pred q, p, 0xffffffff;\n\t}" ::"l"(v) : "memory");
    __syncwarp();
}

template <int LW>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int o = LW / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
template <int LW>
__device__ __forceinline__ float lanes_max(float x) {
#pragma unroll
    for (int o = LW / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// Sums of K (1, 2 or 4) values over the LW lanes of a team, written to out[0..K).
template <int LW, int K>
__device__ __forceinline__ void lanes_sum_to(float (&p)[K], float* out) {
    const int lane = threadIdx.x & 31;
    if constexpr (LW == 32) {  // one lane in 32 / K ends up with one of the sums
        warp_reduce_scatter<K>(p, lane);
        if ((lane & (32 / K - 1)) == 0) out[lane / (32 / K)] = p[0];
    } else {
#pragma unroll
        for (int o = LW / 2; o > 0; o >>= 1) {
#pragma unroll
            for (int i = 0; i < K; ++i) p[i] += __shfl_xor_sync(0xffffffffu, p[i], o);
        }
        if (lane % LW == 0) {
#pragma unroll
            for (int i = 0; i < K; ++i) out[i] = p[i];
        }
    }
}

// A row in a stage: the codes of the warp's 32 threads (16 or 32 bytes each),
// then, after the codes of all rows, the scales and the statistics of its tokens.
template <int BITS, int LW, bool MULTI>
struct RowStage {
    static constexpr int CH = BITS / 4;                 // 16-byte chunks of codes a thread
    static constexpr int TW = 32 / LW;                  // tokens a warp
    static constexpr int SC = LW >= 8 ? 32 : TW * 8;    // scale bytes a row
    static constexpr int ROW = 512 * CH + SC + 8 * TW;  // bytes a row
    __host__ __device__ static int bytes(int seg) { return (seg * ROW + 15) & ~15; }

    // Copies rows s0 .. s0 + cnt - 1 of the warp's tokens (from n0 on; behind
    // the last one the last again) to the stage at shared address `base`;
    // `rows`: the sources' addresses, in shared memory.
    static __device__ __forceinline__ void copy(const CachedArgs& a, const unsigned char* const* rows, uint32_t base,
                                                int seg, long long n0, int s0, int cnt) {
        const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
        long long off[CH];
        bool on[CH];
        uint32_t dst[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = lane + 32 * i;
            const int x = (c % (LW * CH) + (MULTI ? wid * 32 * CH : 0)) * 16;
            on[i] = x < static_cast<int>(a.codes);  // else zeros
            off[i] = min(n0 + c / (LW * CH), a.N - 1) * a.row_ld + (on[i] ? x : 0);
            dst[i] = base + (CH == 2 ? c ^ ((c >> 3) & 1) : c) * 16;  // keeps the 32-byte reads off each other's banks
        }
        for (int r = 0; r < cnt; ++r) {
            const unsigned char* p = rows[s0 + r];
#pragma unroll
            for (int i = 0; i < CH; ++i) cp_async_16z(dst[i] + r * 512 * CH, p + off[i], on[i]);
        }
        const uint32_t sc = base + seg * 512 * CH, stt = sc + seg * SC;
        if constexpr (LW >= 16) {
            constexpr int H = LW / 16;  // chunks of 16 scales a token
            for (int i = lane; i < cnt * TW * H; i += 32) {
                const int r = i / (TW * H), team = i / H % TW, x = (MULTI ? wid * 32 : 0) + i % H * 16;
                if (x < (a.D + 31) / 32)
                    cp_async_16z(sc + r * 32 + team * LW + i % H * 16,
                                 rows[s0 + r] + min(n0 + team, a.N - 1) * a.row_ld + a.codes + x, true);
            }
        } else {
            for (int i = lane; i < cnt * TW; i += 32) {
                const int r = i / TW, team = i % TW;
                cp_async_8s(sc + r * SC + team * 8, rows[s0 + r] + min(n0 + team, a.N - 1) * a.row_ld + a.codes);
            }
        }
        for (int i = lane; i < cnt * TW; i += 32)
            cp_async_8s(stt + i * 8, rows[s0 + i / TW] + min(n0 + i % TW, a.N - 1) * a.row_ld + a.stat);
    }

    // This thread's codes and scale byte: their place in a stage's first row.
    static __device__ __forceinline__ void places(int seg, uint32_t (&code_at)[CH], uint32_t& scale_at) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = lane * CH + i;
            code_at[i] = (CH == 2 ? c ^ ((c >> 3) & 1) : c) * 16;
        }
        scale_at = seg * 512 * CH + (LW >= 8 ? lane : lane / LW * 8 + lane % LW);
    }
    static __device__ __forceinline__ CacheCodes<BITS> codes(uint32_t base, const uint32_t (&code_at)[CH], int r) {
        CacheCodes<BITS> w;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const uint4 u = lds128(base + code_at[i] + r * 512 * CH);
            w.w[4 * i] = u.x, w.w[4 * i + 1] = u.y, w.w[4 * i + 2] = u.z, w.w[4 * i + 3] = u.w;
        }
        return w;
    }
    // A thread without channels reads some other byte: its codes are zero and its sums unused.
    static __device__ __forceinline__ float scale(uint32_t base, uint32_t scale_at, int r) {
        uint32_t b;
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(b) : "r"(base + scale_at + r * SC));
        return cache_scale(b);
    }
    // Mean square and tag of a row for the team `tw` of the warp.
    static __device__ __forceinline__ uint2 stat(uint32_t base, int seg, int r, int tw) {
        uint2 v;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(base + seg * (512 * CH + SC) + (r * TW + tw) * 8));
        return v;
    }

    // A bf16 row per token, 64 bytes a thread; BF16 bytes a warp.
    static constexpr int BF16 = 2048;
    static __device__ __forceinline__ void copy_bf16(const uint16_t* x, long long ld, uint32_t base, long long n0,
                                                     long long N, int D) {
        const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = lane + 32 * i;
            const int at = (c % (LW * 4) + (MULTI ? wid * 128 : 0)) * 8;
            const bool on = at < D;
            cp_async_16z(base + (c ^ ((c >> 3) & 3)) * 16, x + min(n0 + c / (LW * 4), N - 1) * ld + (on ? at : 0), on);
        }
    }
    static __device__ __forceinline__ uint4 bf16_part(uint32_t base, int i) {
        const int c = (threadIdx.x & 31) * 4 + i;
        return lds128(base + (c ^ ((c >> 3) & 3)) * 16);
    }
};

// The same parts of a warp's shared memory filled by bulk copies (teams of
// whole warps): two copies a row instead of an instruction for every 16 bytes
// of each lane.  Nothing is written behind a row's end: a stage starts as
// zeros, so what a row does not have reads as zero.  Statistics are left out.
template <int BITS, bool MULTI>
struct BulkStage {
    static constexpr int CH = BITS / 4;
    static constexpr int ROW = 512 * CH + 32;  // a row's codes; its scales behind the codes of all rows
    __host__ __device__ static int bytes(int seg) { return seg * ROW; }

    const unsigned char* const* rows;
    uint32_t code_from, code_bytes, scale_from, scale_bytes, bf16_from, bf16_bytes;  // of the warp, in a record and in a bf16 row
    int seg;

    __device__ __forceinline__ void init(const CachedArgs& a, const unsigned char* const* table, int rows_a_segment) {
        const uint32_t w = MULTI ? threadIdx.x >> 5 : 0;
        const uint32_t rec = (a.stat + 8 + 15) & ~15u;
        rows = table;
        seg = rows_a_segment;
        code_from = w * 512 * CH;
        code_bytes = min(a.codes - code_from, 512u * CH);
        scale_from = a.codes + w * 32;
        scale_bytes = min(rec - scale_from, 32u);
        bf16_from = w * 1024;  // elements
        bf16_bytes = min((a.D - bf16_from) * 2u, 2048u);
    }
    __device__ __forceinline__ uint32_t row_bytes() const { return code_bytes + scale_bytes; }
    // by one lane
    __device__ __forceinline__ void copy_row(const CachedArgs& a, uint32_t base, long long n, int s, int r, uint32_t bar) const {
        const unsigned char* p = rows[s] + n * a.row_ld;
        bulk_load(base + r * (512 * CH), p + code_from, code_bytes, bar);
        bulk_load(base + seg * (512 * CH) + r * 32, p + scale_from, scale_bytes, bar);
    }
    __device__ __forceinline__ void copy_bf16(const uint16_t* x, uint32_t dst, uint32_t bar) const {
        bulk_load(dst, x + bf16_from, bf16_bytes, bar);
    }
};

// 64 bytes of a thread's bf16 results to global memory: whole 32-byte sectors
// where `wide` (every row starts on a 32-byte boundary and D % 16 == 0).
__device__ __forceinline__ void store_bf16x32(uint16_t* p, int left, bool wide, const uint32_t (&w)[16]) {
    if (wide) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (16 * i < left)
                asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + 16 * i), "r"(w[8 * i]),
                             "r"(w[8 * i + 1]), "r"(w[8 * i + 2]), "r"(w[8 * i + 3]), "r"(w[8 * i + 4]), "r"(w[8 * i + 5]),
                             "r"(w[8 * i + 6]), "r"(w[8 * i + 7])
                             : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (8 * i < left)
                st_global_cs_v4(p + 8 * i, make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
    }
}

// 16 channels to a 32-byte aligned address.
__device__ __forceinline__ void store_half(void* p, bool on, const uint32_t* w) {
    if (on)
        asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
}

// The same from two runs of 16 channels, at channels half[0] and half[1] of a row.
__device__ __forceinline__ void store_halves(uint16_t* row, const int (&half)[2], int D, bool wide, const uint32_t (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint16_t* p = row + half[i];
        if (wide) {
            if (half[i] < D)
                asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[8 * i]),
                             "r"(w[8 * i + 1]), "r"(w[8 * i + 2]), "r"(w[8 * i + 3]), "r"(w[8 * i + 4]), "r"(w[8 * i + 5]),
                             "r"(w[8 * i + 6]), "r"(w[8 * i + 7])
                             : "memory");
        } else {
            if (half[i] < D) st_global_cs_v4(p, make_uint4(w[8 * i], w[8 * i + 1], w[8 * i + 2], w[8 * i + 3]));
            if (half[i] + 8 < D) st_global_cs_v4(p + 8, make_uint4(w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]));
        }
    }
}

}  // namespace attnres
