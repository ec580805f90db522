// Weight-streaming products for a few activation rows (gfx950): the shared
// core of the few-row GroupedLinear and of the few-token MoE layer.
//
// With T rows against an N x K weight the work is 2 T N K operations on
// N K weight values, so up to some 100 rows the time is that of reading the
// weights once.  The weights are the MFMA's first operand (16 rows of W), the
// activations its second (16 columns, one per row of X), so that a wave
// streams weights straight from global memory into operand registers: no LDS
// on the way, no barrier in the loop.  Waves of a workgroup split K (or
// experts) and add their results at the end.
//
// Workgroups are persistent and a wave's weights come as one stream of groups
// over all its units of work, the next group's loads issued before the current
// one is used: a unit's start and end (its plan, its sums) leave no gap in the
// stream.  One wave has 8 or 16 KiB in flight, a CU with eight waves 64 to 128
// KiB, against the some 40 KiB that 5 TB/s times 2 us of loaded latency ask of
// each of 256 CUs.
//
// Fragments.  A lane is (r = lane & 15, q = lane >> 4).  Both operands are
// read in their memory order: 64 bytes of a row per load instruction, lane
// (r, q) taking 16 bytes at 16 q.  128 values of K are one such load for
// MXFP4, two for MXFP8 and four for bf16.  The scaled 16x16x128 MFMA pairs
// the 16 bytes of an E2M1 lane (K values 32 q ..) with the two 16-byte runs of
// an E4M3 lane (16 q .. and 64 + 16 q ..) by K, and takes lane (r, q)'s scale
// as that of K block q of row r (checked on the device with random scales).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "internal.h"
#include "mx_device.h"

namespace mx {
namespace few {

// operand formats
constexpr int kBf16 = 0, kFp8 = 1, kFp4 = 2;

// 16-byte loads a lane makes per row for 128 values of K, and bytes of that row
__host__ __device__ constexpr int loads_per_step(int f) { return f == kFp4 ? 1 : f == kFp8 ? 2 : 4; }
__host__ __device__ constexpr int bytes_per_step(int f) { return 64 * loads_per_step(f); }
// bytes of a row of K values
__host__ __device__ constexpr int64_t row_bytes(int f, int64_t K) {
    return f == kFp4 ? K / 2 : f == kFp8 ? K : 2 * K;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_a4 __attribute__((ext_vector_type(2), aligned(4)));

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The operand registers of one 128-value step of one 16-row tile.
template <int F>
__device__ __forceinline__ v8i mx_frag(const u32x4* c) {
    if constexpr (F == kFp4)
        return v8i{(int)c[0].x, (int)c[0].y, (int)c[0].z, (int)c[0].w, 0, 0, 0, 0};
    else
        return v8i{(int)c[0].x, (int)c[0].y, (int)c[0].z, (int)c[0].w,
                   (int)c[1].x, (int)c[1].y, (int)c[1].z, (int)c[1].w};
}

template <int WF, int XF>
__device__ __forceinline__ v4f mac_step(v4f acc, const u32x4* w, uint32_t ws, const u32x4* x, uint32_t xs) {
    if constexpr (WF == kBf16) {
        static_assert(XF == kBf16, "bf16 weights take bf16 activations");
#pragma unroll
        for (int l = 0; l < 4; ++l)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[l]),
                                                          __builtin_bit_cast(bf16x8, x[l]), acc, 0, 0, 0);
        return acc;
    } else {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            mx_frag<WF>(w), mx_frag<XF>(x), acc, WF == kFp4 ? 4 : 0, XF == kFp4 ? 4 : 0, 0, (int)ws, 0,
            (int)xs);
    }
}

// A lane's place in a 16-row tile: byte offsets of its row's codes (at its 16
// bytes of K = 0) and scales from the tile's first row.
struct LaneRow {
    uint32_t codes, scales;
    int q;
};
template <int F>
__device__ __forceinline__ LaneRow lane_row(int64_t K, int lane) {
    return LaneRow{(uint32_t)((lane & 15) * row_bytes(F, K)) + (uint32_t)(lane >> 4) * 16u,
                   (uint32_t)((lane & 15) * (K / 32)), lane >> 4};
}

// kSteps consecutive 128-value steps of one tile in registers, from the tile's
// first row (codes, scales: wave-uniform for weights, a lane's own row with a
// zero LaneRow for activations).  Steps at or past `last` (uniform) repeat step
// last - 1 and are skipped by the caller: the loads stay in range without a
// branch per lane.
// ODD (K % 128 != 0; MX formats): 16-byte chunks past K read as zero codes,
// their scales as 2^0, and scales are read byte by byte (their rows start at
// any byte).
template <int F, int kSteps, bool ODD>
struct Tile {
    static constexpr int kL = loads_per_step(F);
    u32x4 c[kSteps * kL];
    uint32_t s[F == kBf16 ? 1 : kSteps];     // 4 blocks' scales (ODD: this lane's alone)

    __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, const LaneRow& r,
                                         int step, int last, int64_t K) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int st = min(step + i, last - 1);
#pragma unroll
            for (int l = 0; l < kL; ++l) {
                const uint8_t* p = codes + (int64_t)st * bytes_per_step(F) + l * 64 + r.codes;
                if constexpr (ODD) {
                    // first value of the chunk: E2M1 16 bytes are 32 values, E4M3 16
                    const int64_t k0 = (int64_t)st * 128 + (F == kFp4 ? r.q * 32 : l * 64 + r.q * 16);
                    c[i * kL + l] = u32x4{0, 0, 0, 0};
                    if (k0 < K) c[i * kL + l] = *reinterpret_cast<const u32x4*>(p);
                } else {
                    c[i * kL + l] = *reinterpret_cast<const u32x4*>(p);
                }
            }
        }
        if constexpr (F == kBf16) {
        } else if constexpr (ODD) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int st = min(step + i, last - 1);
                s[i] = 127;
                if ((int64_t)st * 128 + r.q * 32 < K) s[i] = scales[(int64_t)st * 4 + r.q + r.scales];
            }
        } else if (kSteps % 2 == 0 && step + kSteps <= last) {
            const uint8_t* p = scales + (int64_t)step * 4 + r.scales;
            if constexpr (kSteps % 4 == 0) {
#pragma unroll
                for (int i = 0; i + 3 < kSteps; i += 4) {
                    const u32x4 v = *reinterpret_cast<const u32x4_a4*>(p + i * 4);
                    s[i] = v.x;
                    s[i + 1] = v.y;
                    s[i + 2] = v.z;
                    s[i + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i + 1 < kSteps; i += 2) {
                    const auto v = *reinterpret_cast<const u32x2_a4*>(p + i * 4);
                    s[i] = v.x;
                    s[i + 1] = v.y;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
                s[i] = *reinterpret_cast<const uint32_t*>(scales + (int64_t)min(step + i, last - 1) * 4 + r.scales);
        }
    }
    // the scale operand of step i: this lane's block in the low byte
    __device__ __forceinline__ uint32_t scale(int i, int q) const {
        if constexpr (F == kBf16) return 0;
        else if constexpr (ODD) return s[i];
        else return s[i] >> (8 * q);
    }
};

// An activation row as a lane reads it: its 16 bytes of K = 0 and its scales.
struct XRow {
    const uint8_t* codes;
    const uint8_t* scales;
};
template <int F>
__device__ __forceinline__ XRow x_row(const uint8_t* codes, const uint8_t* scales, int64_t row, int64_t K,
                                      int lane) {
    return XRow{codes + row * row_bytes(F, K) + (lane >> 4) * 16,
                F == kBf16 ? nullptr : scales + row * (K / 32)};
}

// One unit of a wave's work, all of it wave-uniform: RT tiles of weights (their
// first rows), `rows` activation rows in NT tiles, steps [s0, s1) of K (at least
// one).  id and row0 are the caller's.
template <int RT>
struct Unit {
    const uint8_t* wc[RT];
    const uint8_t* ws[RT];
    int64_t row0;
    int rows, s0, s1, id;
};

// The products of all of a wave's units: first(u) gives the first one, next(u)
// the one after u (false: no more), xrow(u, n) a lane's activation row of tile n
// (rows past u.rows: any valid one, their products go nowhere), ending(u) is
// called before a unit's last loads and done(acc, u) takes its sums: what done
// needs from global memory is loaded in ending, since a load issued in done would
// wait for the next unit's weights.
// A wave's loads return in the order they were issued, so what a group's
// products need is issued before the next group's weights: its activation rows
// too (from the L2), for as many of their tiles as the registers hold, skipping
// tiles without rows.  (Issued after them, the rows waited for the next weights
// and the stream lost its overlap.)
template <int WF, int XF, int RT, int NT, int kSteps, bool ODD, class First, class Next, class XRowOf,
          class Ending, class Done>
__device__ __forceinline__ void stream(int64_t K, int lane, First first, Next next, XRowOf xrow,
                                       Ending ending, Done done) {
    using U = Unit<RT>;
    using TW = Tile<WF, kSteps, ODD>;
    using TX = Tile<XF, kSteps, ODD>;
    // registers: two groups of weights, the sums, and kFirst tiles of X, of the
    // 256 that two waves a SIMD have
    constexpr int kHeld = 2 * RT * kSteps * (4 * TW::kL + 1) + 4 * RT * NT, kX = kSteps * (4 * TX::kL + 1);
    constexpr int kFirst = (232 - kHeld) / kX >= NT ? NT : (232 - kHeld) / kX;
    static_assert(kFirst >= 1 && NT <= 4, "a group of weights and a tile of rows fit");
    struct Group {
        TW w[RT];
    };
    const LaneRow lr = lane_row<WF>(K, lane);
    const LaneRow own{0u, 0u, lane >> 4};      // x rows are the lanes' own
    const int q = lane >> 4;
    v4f acc[RT][NT];
    auto clear = [&]() {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[t][n] = v4f{0.f, 0.f, 0.f, 0.f};
    };
    auto load = [&](Group& g, const U& u, int step) {
#pragma unroll
        for (int t = 0; t < RT; ++t) g.w[t].load(u.wc[t], u.ws[t], lr, step, u.s1, K);
    };
    auto mac = [&](const Group& g, const TX& x, auto nc, const U& u, int step) {
        constexpr int n = decltype(nc)::value;
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            if (i == 0 || step + i < u.s1) {
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    acc[t][n] = mac_step<WF, XF>(acc[t][n], g.w[t].c + i * TW::kL, g.w[t].scale(i, q),
                                                 x.c + i * TX::kL, x.scale(i, q));
            }
    };
    TX xs[kFirst];
    auto load_x = [&](TX& x, const U& u, int n, int step) {
        const XRow r = xrow(u, n);
        x.load(r.codes, r.scales, own, step, u.s1, K);
    };
    // f(integral_constant<n>) for the tiles A <= n < B that have rows
    auto tiles = [&](auto ac, auto bc, const U& u, auto&& f) {
        auto one = [&](auto nc) {
            constexpr int n = decltype(nc)::value;
            if constexpr (n >= decltype(ac)::value && n < decltype(bc)::value)
                if (n == 0 || n * 16 < u.rows) f(nc);
        };
        one(std::integral_constant<int, 0>{});
        one(std::integral_constant<int, 1>{});
        one(std::integral_constant<int, 2>{});
        one(std::integral_constant<int, 3>{});
    };
    constexpr std::integral_constant<int, 0> k0{};
    constexpr std::integral_constant<int, kFirst> kF{};
    constexpr std::integral_constant<int, NT> kN{};
    U u;
    if (!first(u)) return;
    int step = u.s0;
    Group a, b;
    clear();
    load(a, u, step);
    // one turn: the next group's loads, then this one's products
    auto turn = [&](Group& mine, Group& other) -> bool {
        U v = u;
        int vstep = step + kSteps;
        bool more = true;
        if (vstep >= u.s1) {
            more = next(v);
            vstep = v.s0;
        }
        if (step + kSteps >= u.s1) ending(u);
        tiles(k0, kF, u, [&](auto nc) { load_x(xs[decltype(nc)::value], u, decltype(nc)::value, step); });
        if (more) load(other, v, vstep);
        tiles(k0, kF, u, [&](auto nc) { mac(mine, xs[decltype(nc)::value], nc, u, step); });
        tiles(kF, kN, u, [&](auto nc) {
            TX x;
            load_x(x, u, decltype(nc)::value, step);
            mac(mine, x, nc, u, step);
        });
        if (step + kSteps >= u.s1) {
            done(acc, u);
            clear();
        }
        u = v;
        step = vstep;
        return more;
    };
    while (turn(a, b) && turn(b, a)) {
    }
}

}  // namespace few
}  // namespace mx
