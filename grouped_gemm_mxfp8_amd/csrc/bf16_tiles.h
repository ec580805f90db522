// Device helpers of the bf16 tile products (gfx950): operands staged in LDS by
// direct loads, read as fragments of the 32x32x16 MFMA, and the stores of its
// accumulators.
//
// An operand of a product lies in memory in one of two ways:
//   along K:   rows of the output dimension, K contiguous (x and w of a forward).
//              Staged as 128-byte lines of 64 K values, fragments by 16-byte
//              reads.
//   across K:  rows of K, the output dimension contiguous (w of a data gradient,
//              both operands of a weight gradient).  Staged as it lies, 64 rows
//              of K, fragments by the transposing LDS read: 16 lanes fetch four
//              rows of 16 values, 8 bytes a lane, and lane i receives the four
//              values of column i.
//
// MFMA fragments: lane l holds row (or column) l & 31 of a block of 32 and K
// values 8 (l >> 5) .. + 7 of 16.  The column operand goes first, so lane l of an
// accumulator holds output row l & 31 and columns 8 (v >> 2) + 4 (l >> 5) + (v & 3),
// v = 0 .. 15.
#pragma once
#include "gemm_device.h"

namespace mx {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));

template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ v16f zero16() {
    return v16f{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
}

__device__ __forceinline__ v16f mfma_bf16(const bf16x8& cols, const bf16x8& rows, const v16f& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(cols, rows, c, 0, 0, 0);
}

// ---- tiles ------------------------------------------------------------------------
// Groups of rows [offs[g], offs[g + 1]) in tiles of BM rows, group after group: how many
// tiles there are, and the group of one.  A wave does this with a lane per group.
template <int BM>
__device__ __forceinline__ int row_tiles(int64_t beg, int64_t end) {
    return end > beg ? (int)((end - beg + BM - 1) / BM) : 0;
}
__device__ __forceinline__ int wave_prefix(int v, int lane) {          // inclusive
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}
template <int BM>
__device__ __forceinline__ int count_row_tiles(const int64_t* offs, int G, int lane) {
    int n = 0;
    for (int c = 0; c < G; c += 64)
        if (c + lane < G) n += row_tiles<BM>(offs[c + lane], offs[c + lane + 1]);
#pragma unroll
    for (int d = 32; d; d >>= 1) n += __shfl_xor(n, d);
    return uni(n);
}
struct RowGroup {
    int g, first, tiles;      // group (-1: there is no such tile), its first tile, how many it has
    int64_t row0, rows;
};
template <int BM>
__device__ __forceinline__ RowGroup find_row_group(const int64_t* offs, int G, int tile, int lane) {
    int base = 0;
    for (int c = 0; c < G; c += 64) {
        const int g = c + lane;
        const int64_t beg = g < G ? offs[g] : 0, end = g < G ? offs[g + 1] : 0;
        const int cnt = row_tiles<BM>(beg, end), incl = base + wave_prefix(cnt, lane);
        const uint64_t after = __ballot(incl > tile);
        if (after) {
            const int l = __builtin_ctzll(after);
            auto at = [&](int64_t v) {
                const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, l);
                const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)v >> 32), l);
                return (int64_t)(((uint64_t)hi << 32) | lo);
            };
            const int n = __builtin_amdgcn_readlane(cnt, l);
            const int64_t row0 = at(beg);
            return RowGroup{uni(c + l), __builtin_amdgcn_readlane(incl, l) - n, n, row0, at(end) - row0};
        }
        base = __builtin_amdgcn_readlane(incl, 63);
    }
    return RowGroup{-1, 0, 0, 0, 0};
}

// The large kernel's order of a group's tiles: bands of BAND row tiles, so that the tiles
// an XCD runs together share panels of both operands in its L2.
constexpr int BAND = 8;
struct TileAt {
    int m, n;
};
__device__ __forceinline__ TileAt band_order(int local, int mtiles, int ntn) {
    const int band = local / (BAND * ntn);
    const int rem = local - band * BAND * ntn;
    const int bm = min(BAND, mtiles - band * BAND);
    return TileAt{band * BAND + rem % bm, rem / bm};
}

// Rounds of the large kernel.  It runs `grid` tiles at a time; a last round of up to
// kTailMost tiles is left to the middle tiles, four to a large one, two at a time on a CU.
constexpr int kTailMost = 176;
__device__ __host__ __forceinline__ int whole_rounds(int tiles, int grid) {
    const int rest = tiles % grid;
    return rest <= kTailMost ? tiles - rest : tiles;
}

// Fragment of an operand staged along K: 16 bytes.
__device__ __forceinline__ bf16x8 frag_along(const uint8_t* p) {
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4*>(p));
}

// Fragment of an operand staged across K: two transposing reads, K values 0..3 at
// p and 4..7 four rows on.  p is the lane's own 8 bytes: row (l >> 2) & 3 of the
// four, columns 16 ((l >> 4) & 1) + 4 (l & 3) of the block.
__device__ __forceinline__ bf16x8 frag_across(const uint8_t* p, int four_rows) {
    typedef __attribute__((address_space(3))) v4s* lds_v4s;
    struct Pair {
        v4s a, b;
    } v;
    v.a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p));
    v.b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p + four_rows));
    return __builtin_bit_cast(bf16x8, v);
}

// ---- stores ---------------------------------------------------------------------
// Values of 32 rows, 16 bytes (four dwords) of each line segment S = 0 .. 3 and
// half l >> 5 in lane l of row l & 31, moved so that store T = 0 .. 3 writes whole
// 128-byte lines of rows 8 T .. 8 T + 7: lane l then holds row 8 T + (l & 7),
// 16-byte chunk 2 S + (l >> 5) with S = 2 (l >> 4 & 1) + (l >> 3 & 1).  A 4 x 4
// transposition of S against the row's bits 4 and 3: one swap of 16-lane rows, one
// rotation by 8 within them.
__device__ __forceinline__ void to_lines(uint32_t (&x)[4][4]) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const auto z = __builtin_amdgcn_permlane16_swap(x[s][v], x[s + 2][v], false, false);
            x[s][v] = z[0];
            x[s + 2][v] = z[1];
        }
#pragma unroll
    for (int s = 0; s < 4; s += 2)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const uint32_t a = x[s][v], b = x[s + 1][v];
            // lanes 8..15 of each 16 take b of lane ^ 8, lanes 0..7 a of lane ^ 8
            x[s][v] = (uint32_t)__builtin_amdgcn_update_dpp((int)a, (int)b, 0x128, 0xf, 0xc, false);
            x[s + 1][v] = (uint32_t)__builtin_amdgcn_update_dpp((int)b, (int)a, 0x128, 0xf, 0x3, false);
        }
}
__device__ __forceinline__ int line_chunk(int lane) {
    return 4 * (lane >> 4 & 1) + 2 * (lane >> 3 & 1) + (lane >> 5);
}

// 32 rows x 64 columns (two accumulators) as bf16 lines.  base: row 0, column 0
// (wave-uniform), ldb: bytes between rows; rows and cols: how many of them exist
// (cols a multiple of 8).  sc: the factor of row lane & 31.  MAPPED: base is row 0 of the
// matrix and at[t] the row that store t's row 8 t + (lane & 7) belongs at.
template <bool SCALED, bool MAPPED = false>
__device__ __forceinline__ void store_bf16_32x64(const v16f& a0, const v16f& a1, float sc, uint8_t* base,
                                                 uint32_t ldb, int rows, int cols, int lane,
                                                 const int (&at)[4] = {0, 0, 0, 0}) {
    uint32_t x[4][4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const v16f& a = s < 2 ? a0 : a1;
        const int p = 8 * (s & 1);
        float va[4], vb[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            va[v] = SCALED ? a[p + v] * sc : a[p + v];
            vb[v] = SCALED ? a[p + 4 + v] * sc : a[p + 4 + v];
        }
        const uint2 lo = pack4_bf16(va), hi = pack4_bf16(vb);
        const auto y = __builtin_amdgcn_permlane32_swap(lo.x, hi.x, false, false);
        const auto z = __builtin_amdgcn_permlane32_swap(lo.y, hi.y, false, false);
        x[s][0] = y[0];
        x[s][1] = z[0];
        x[s][2] = y[1];
        x[s][3] = z[1];
    }
    to_lines(x);
    const int r8 = lane & 7, chunk = line_chunk(lane);
    const uint32_t off = (uint32_t)r8 * ldb + (uint32_t)chunk * 16u;
    if (chunk * 8 < cols) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (8 * t + r8 < rows)
                store_nt(MAPPED ? base + (int64_t)at[t] * ldb + (uint32_t)chunk * 16u
                                : base + (int64_t)(8 * t) * ldb + off,
                         make_uint4(x[t][0], x[t][1], x[t][2], x[t][3]));
    }
}

// Where the rows of a block's four stores belong (its row 0 is row r0): order's, or as
// they are.
__device__ __forceinline__ void line_rows(int (&at)[4], const int32_t* order, int64_t r0, int rows, int lane) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int r = 8 * t + (lane & 7);
        at[t] = order ? (r < rows ? order[r0 + r] : 0) : (int)(r0 + r);
    }
}

// 32 rows x 32 columns (one accumulator) as fp32 lines (cols a multiple of 4).
// ADD: added to what is there.
template <bool ADD>
__device__ __forceinline__ void store_f32_32x32(const v16f& a, uint8_t* base, int64_t ldb, int rows,
                                                int cols, int lane) {
    uint32_t x[4][4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int v = 0; v < 4; ++v) x[s][v] = __float_as_uint(a[4 * s + v]);
    to_lines(x);
    const int r8 = lane & 7, chunk = line_chunk(lane);
    if (chunk * 4 < cols) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (8 * t + r8 < rows) {
                uint4* const at = reinterpret_cast<uint4*>(base + (8 * t + r8) * ldb + chunk * 16);
                uint4 y = make_uint4(x[t][0], x[t][1], x[t][2], x[t][3]);
                if constexpr (ADD) {
                    const float4 o = *reinterpret_cast<const float4*>(at);
                    y = make_uint4(__float_as_uint(o.x + __uint_as_float(y.x)),
                                   __float_as_uint(o.y + __uint_as_float(y.y)),
                                   __float_as_uint(o.z + __uint_as_float(y.z)),
                                   __float_as_uint(o.w + __uint_as_float(y.w)));
                }
                store_nt(at, y);
            }
    }
}

// Sum over a block's 32 columns of accumulator times x of the same rows and columns
// (lane l: its half of row l & 31).  xr: x at the row's first column of the block,
// null for a row that does not exist; cols as above, a multiple of 16.
__device__ __forceinline__ float dot_32(const v16f& a, const uint16_t* xr, int cols, int lane) {
    const int half = lane >> 5;
    float sum = 0.f;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        if (16 * p >= cols) continue;       // (accumulators past the columns may hold anything)
        uint4 d = make_uint4(0, 0, 0, 0);
        if (xr) d = *reinterpret_cast<const uint4*>(xr + 16 * p + 8 * half);
        // 8 consecutive columns a lane to the accumulator's 4 + 4
        const auto u = __builtin_amdgcn_permlane32_swap(d.x, d.z, false, false);
        const auto w = __builtin_amdgcn_permlane32_swap(d.y, d.w, false, false);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int v = 8 * p + 4 * g;
            sum += a[v] * bf16_to_f32(u[g] & 0xffffu) + a[v + 1] * __uint_as_float(u[g] & 0xffff0000u);
            sum += a[v + 2] * bf16_to_f32(w[g] & 0xffffu) + a[v + 3] * __uint_as_float(w[g] & 0xffff0000u);
        }
    }
    return sum;
}

// The adapters' part of 32 rows x 32 NB columns, added to the accumulators of the
// rows' own adapters: h b^T with h as two bf16 values (hi + lo) a number.  lane l:
// row l & 31, id its adapter or negative, hrow its h (hi values, then lo values,
// r each; null for a row that does not exist).  b: [.][N][r]; col: the wave's first
// column.  Each adapter among the rows is multiplied for itself, sixteen ranks at a
// time from zero, and only its own rows take the result: what another adapter's
// weights hold, NaN included, never meets a row.  U products' operands are in flight
// together (one by one, 32 rows of 32 adapters took 16 us of loads' latency).
template <int NB, int U>
__device__ __forceinline__ void add_adapters(v16f (&acc)[NB], const LowRank& lr, const uint16_t* hrow, int id,
                                             int64_t N, int64_t col, int lane) {
    const int half = lane >> 5, r = lr.r;
    uint64_t left = __ballot(hrow != nullptr && id >= 0);
    int k = 0;
    while (left) {
        uint4 hi[U], lo[U], bv[U][NB];
        int who[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            who[u] = -1;
            if (left == 0) continue;
            const int one = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
            who[u] = one;
            const bool mine = hrow != nullptr && id == one;
            const int kl = k + 8 * half;
            hi[u] = lo[u] = make_uint4(0, 0, 0, 0);
            if (mine && kl < r) {
                hi[u] = *reinterpret_cast<const uint4*>(hrow + kl);
                lo[u] = *reinterpret_cast<const uint4*>(hrow + r + kl);
            }
            const uint16_t* const b = lr.b + (int64_t)one * N * r + kl;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int64_t n = col + 32 * j + (lane & 31);
                bv[u][j] = make_uint4(0, 0, 0, 0);
                if (n < N && kl < r) bv[u][j] = *reinterpret_cast<const uint4*>(b + n * r);
            }
            k += 16;
            if (k >= r) {
                k = 0;
                left &= ~__ballot(mine);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (who[u] < 0) continue;
            v16f t[NB];
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const bf16x8 bf = __builtin_bit_cast(bf16x8, bv[u][j]);
                t[j] = mfma_bf16(bf, __builtin_bit_cast(bf16x8, hi[u]), zero16());
                t[j] = mfma_bf16(bf, __builtin_bit_cast(bf16x8, lo[u]), t[j]);
            }
            if (hrow != nullptr && id == who[u]) {
#pragma unroll
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int v = 0; v < 16; ++v) acc[j][v] += t[j][v];
            }
        }
    }
}

}  // namespace
}  // namespace mx
