// The adapters' down projection (gfx950): h[m] = scale[l] x[m] a[l]^T with l the
// adapter of row m, stored as the high and the low bf16 part of each fp32 value (the
// sum of both is off by at most 2^-16 of it, so the product with b that follows
// loses nothing a bf16 result could show).
//
// A workgroup of eight waves takes 16 rows and 16 ranks.  Where the rows have one or
// two adapters, as in a prompt, they are multiplied on the MFMA, one adapter after the
// other, the waves sharing K.  Where they have more, as decoded tokens do, pairs of
// waves take a row and four ranks of its own adapter as dot products, so that the work
// is the same however many adapters there are (16 rows of 16 adapters, r = 64, K =
// 4096: one adapter after the other on the MFMA 106 us).  Those dots are spread over
// sixteen workgroups in calls small enough for that to fill the GPU (FINE).
//
// Calls of many rows sort them by adapter first, so that here and in the product's
// tiles most blocks of rows have one adapter whatever the batch's order.  Many of those take
// the tiles of a product instead (bf16_down_kernel), which read x once for 128 ranks.
#pragma once
#include "bf16_tiles.h"

namespace mx {
namespace {

// Rows times ranks up to which the dots are spread: 4096 workgroups, of which a prompt's
// blocks use one in sixteen or 32.
constexpr int64_t kDownFine = 65536;

// Rows times ranks past which sorted rows take tiles of 64 rows x 128 ranks, though the ranks
// fill few of the 128: a tile of 64 steps in K takes 26 us however full.  The whole call at 16
// adapters, K x N = 4096 x 1024, us without tiles and with: 1003 rows of rank 64 50.9 and 51.3,
// 5001 of rank 16 81.9 and 83.1, of 32 92.3 and 84.9, 16384 rows of rank 16 179 and 177, of 64
// 281 and 197, of 128 421 and 230.
constexpr int64_t kDownTiles = 131072;

// The two bf16 parts of f.  A finite value past bf16's largest, which rounding would make an
// infinity, is cut off instead: its rest is below 2^-7 of it, and with it the two are off by at
// most 2^-16 as elsewhere.  (An infinity has no rest: inf - inf would make it a NaN.)
__device__ __forceinline__ void split2(float f, uint32_t& hi, uint32_t& lo) {
    hi = f32_to_bf16(f);
    if ((hi & 0x7fffu) == 0x7f80u && __builtin_isfinite(f)) hi = __float_as_uint(f) >> 16;
    const float rest = f - bf16_to_f32(hi);
    lo = __builtin_isfinite(rest) ? f32_to_bf16(rest) : 0u;
}

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float s) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s += bf16_to_f32(x[i] & 0xffffu) * bf16_to_f32(y[i] & 0xffffu);
        s += __uint_as_float(x[i] & 0xffff0000u) * __uint_as_float(y[i] & 0xffff0000u);
    }
    return s;
}

__device__ __forceinline__ float dot8f(const float (&h)[8], const uint4& b, float s) {
    const uint32_t y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s += h[2 * i] * bf16_to_f32(y[i] & 0xffffu);
        s += h[2 * i + 1] * __uint_as_float(y[i] & 0xffff0000u);
    }
    return s;
}

// The part of workgroup (bx, by, bz) of (rows / 16, ..): WAVES waves, 16 RB ranks on the
// MFMA.
template <int WAVES, int RB, bool FINE>
__device__ __forceinline__ void lora_down(const LoraDown& p, const int bx, const int by, const int bz,
                                          v4f (&s_sum)[WAVES][RB][64]) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int r16 = lane & 15, q = lane >> 4, r = p.r;
    const int64_t row0 = (int64_t)bx * 16, row = row0 + r16, M = p.M, K = p.K;
    int id = row < M ? p.ids[row] : -1;
    if (id >= p.L) id = -1;
    const float sc = p.scale && id >= 0 ? p.scale[id] : 1.f;
    uint64_t left = __ballot(id >= 0);
    int kinds = 0;                                // adapters among the rows, up to three
    for (uint64_t m = left; m && kinds < 3; ++kinds)
        m &= ~__ballot(id == __builtin_amdgcn_readlane(id, __builtin_ctzll(m)));
    // (a row's scale and parts: what lane (r16, q) holds of its row's four ranks)
    auto store = [&](const v4f& v, float by_, int64_t to, int rank) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2(v[e] * by_, hi[e], lo[e]);
        uint16_t* const at = p.h + to * (2 * r) + rank;
        *reinterpret_cast<uint2*>(at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
        *reinterpret_cast<uint2*>(at + r) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
    };

    // Spread dots also serve a block with few rows: one adapter on the MFMA takes a workgroup
    // 7 us (K = 4096) however few there are.  The two add in different orders, so the last bits of
    // a row's h go by the adapters beside it.  (Sorted rows always go to the MFMA: a row's sums are
    // then the same whatever rows are beside it, and with them the same for any order among an
    // adapter's rows.)
    if (!p.order && (kinds > 2 || (FINE && __popcll(left) <= 32))) {
        // FINE: by counts ranks in fours, bz rows in fours; else ranks in 16 RB, all rows
        constexpr int RANKS = FINE ? 4 : 16 * RB, PARTS = WAVES / 4;
        if (!FINE && bz) return;
        const int rank_beg = by * RANKS, rank_end = min(r, rank_beg + RANKS);
        const int row_beg = FINE ? bz * 4 : 0, row_end = FINE ? row_beg + 4 : 16;
        const int part = wave % PARTS;            // of K: 512 values in turn
        for (int rb = row_beg; rb < row_end; rb += 4) {
            const int mine = rb + wave / PARTS;
            const int own = __builtin_amdgcn_readlane(id, mine);
            const float by_ = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(sc), mine));
            const uint16_t* const xr = p.x + min(row0 + mine, M - 1) * K;
            for (int rank = rank_beg; rank < rank_end; rank += 4) {
                v4f s = {0.f, 0.f, 0.f, 0.f};
                if (own >= 0) {
                    const uint16_t* const ar = p.a + ((int64_t)own * r + rank) * K;
                    // twenty loads in flight
                    for (int64_t k0 = part * 512 + lane * 8; k0 - lane * 8 < K; k0 += 2048 * PARTS) {
                        uint4 xv[4], av[4][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int64_t k = k0 + i * 512 * PARTS, kc = k < K ? k : K - 8;
                            xv[i] = *reinterpret_cast<const uint4*>(xr + kc);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                av[i][e] = *reinterpret_cast<const uint4*>(ar + e * K + kc);
                        }
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (k0 + i * 512 * PARTS < K)
#pragma unroll
                                for (int e = 0; e < 4; ++e) s[e] = dot8(xv[i], av[i][e], s[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int d = 32; d; d >>= 1) s[e] += __shfl_xor(s[e], d);
                }
                if constexpr (PARTS > 1) {
                    if (lane == 0) s_sum[wave][0][0] = s;
                    __syncthreads();
                    if (part == 0) s = s_sum[wave][0][0] + s_sum[wave + 1][0][0];
                    __syncthreads();
                }
                if (own >= 0 && part == 0 && lane == 0) store(s, by_, row0 + mine, rank);
            }
        }
        return;
    }

    if (FINE && (by % (4 * RB) || bz)) return;
    const int rank0 = by * (FINE ? 4 : 16 * RB);
    const int64_t in = row < M ? row : M - 1;
    const uint16_t* const xr = p.x + (p.order ? p.order[in] : in) * K;
    // K in steps of 64, two MFMAs; a load takes 64 consecutive bytes of each row.  The last
    // step may have 32 values: its second load takes the last ones again, as zeros
    const int nk = (int)((K + 63) / 64);
    const int k_beg = nk * wave / WAVES, k_end = nk * (wave + 1) / WAVES;
    for (int turn = 0; left; ++turn) {
        const int one = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        if (!FINE && (turn & 1) != bz) {          // bz: even and odd ones
            left &= ~__ballot(id == one);
            continue;
        }
        const uint16_t* ar[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) {            // (ranks past r read the first one's row)
            const int rank = rank0 + 16 * b + r16;
            ar[b] = p.a + ((int64_t)one * r + (rank < r ? rank : 0)) * K;
        }
        v4f acc[RB][2];
#pragma unroll
        for (int b = 0; b < RB; ++b) acc[b][0] = acc[b][1] = v4f{0.f, 0.f, 0.f, 0.f};
        auto steps = [&](auto nc, int ks) {       // n steps, their loads in flight together
            constexpr int n = decltype(nc)::value;
            uint4 xv[n][2], av[n][2][RB];
#pragma unroll
            for (int i = 0; i < n; ++i) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int64_t k = min((int64_t)(ks + i) * 64 + u * 32, K - 32) + q * 8;
                    xv[i][u] = *reinterpret_cast<const uint4*>(xr + k);
#pragma unroll
                    for (int b = 0; b < RB; ++b) av[i][u][b] = *reinterpret_cast<const uint4*>(ar[b] + k);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < n; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const bool live = (int64_t)(ks + i) * 64 + u * 32 < K;
                    const uint4 z = make_uint4(0, 0, 0, 0);
                    const bf16x8 xz = __builtin_bit_cast(bf16x8, live ? xv[i][u] : z);
#pragma unroll
                    for (int b = 0; b < RB; ++b)
                        acc[b][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, live ? av[i][u][b] : z), xz, acc[b][u], 0, 0, 0);
                }
        };
        int ks = k_beg;
        for (; ks + 4 <= k_end; ks += 4) steps(std::integral_constant<int, 4>{}, ks);
        if (ks + 2 <= k_end) steps(std::integral_constant<int, 2>{}, ks), ks += 2;
        if (ks < k_end) steps(std::integral_constant<int, 1>{}, ks);
        // lane (r16, q): row r16, ranks 4 q .. + 3
#pragma unroll
        for (int b = 0; b < RB; ++b) s_sum[wave][b][lane] = acc[b][0] + acc[b][1];
        __syncthreads();
        if (wave < RB && id == one && rank0 + 16 * wave + 4 * q < r) {
            v4f v = s_sum[0][wave][lane];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) v += s_sum[w][wave][lane];
            store(v, sc, row, rank0 + 16 * wave + 4 * q);
        }
        __syncthreads();
        left &= ~__ballot(id == one);
    }
}

}  // namespace
}  // namespace mx
