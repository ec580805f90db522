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
//
// Precision.  The sums are fp32, but with an E4M3 operand that MFMA first cuts
// the eight products of each run of eight K values to multiples of 2^-13 of
// their largest (E2M1 x E2M1 products span less than that and lose nothing).
// The GroupedLinear takes that, as every MXFP8 product of the library: its bf16
// result is coarser by far, except where large products cancel.  The layer does
// not: z is quantized from its first sums, and at K = 2048 the cut put those off
// by 2e-5 to 6e-5 of themselves, which moved large values of z by whole E4M3
// steps (out off by up to 3.0e-3 in norm, the rounding of out alone 1.7e-3).
// Its products are exact: operands converted to bf16 in registers, on the bf16
// MFMA (out off by 1.7e-3, bit for bit an fp32 sum's in most cases).  The
// conversions cost 1 to 2 % of the layer's time with MXFP8 weights and 2 to 8 %
// with MXFP4 (1 token, 8 x (4096, 14336): 48.4 -> 51.6 us; 64 tokens 208 -> 211;
// 64 x (2048, 1408), 16 tokens: 73.1 -> 78.3).
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

// Exact products of MX operands: the values that codes and scales stand for, as
// bf16 (at most 4 significant bits; exact from 2^-126 up, and past bf16's largest,
// which no quantizer's blocks reach, infinity), on the bf16 MFMA, whose products
// and sums are fp32.  Its 32 values of K are four times eight, lane (r, q) holding
// eight of row r: any eight, as long as both operands hold the same.

typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));

// The scale of byte b of s, an E8M0 code, as the conversions take it: its bits as
// an fp32 exponent.  (They read exponent 0 as 2^-127 and 255 as NaN, whatever the
// code: checked on the device for every code and scale.)
__device__ __forceinline__ float block_scale(uint32_t s, int b) {
    return __uint_as_float(__builtin_amdgcn_ubfe(s, 8 * b, 8) << 23);
}

// Eight values of a lane's chunk j (of four) of a step as bf16.  c: the step's
// codes, s: the scale of the chunk's block.  MXFP4: dword j of the lane's 32
// values.  MXFP8: dwords 2 j and 2 j + 1.
template <int F>
__device__ __forceinline__ bf16x8 exact_chunk(const u32x4* c, float s, int j) {
    uint32_t v[4];
    auto put = [&](int i, const bf16x2v& p) { v[i] = __builtin_bit_cast(uint32_t, p); };
    if constexpr (F == kFp4) {
        const uint32_t d = c[0][j];
        put(0, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 0));
        put(1, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 1));
        put(2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 2));
        put(3, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 3));
    } else {
        const int a = (int)c[j >> 1][2 * (j & 1)], b = (int)c[j >> 1][2 * (j & 1) + 1];
        put(0, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, false));
        put(1, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, true));
        put(2, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, false));
        put(3, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, true));
    }
    return __builtin_bit_cast(bf16x8, u32x4{v[0], v[1], v[2], v[3]});
}
// The scale of chunk j, s: the step's four.  Where both operands are MXFP8 a lane
// holds K values 16 q .. and 64 + 16 q .., of blocks q / 2 and 2 + q / 2; MXFP4
// weights and rows beside them (RUN) 32 q .., of block q.
template <bool RUN>
__device__ __forceinline__ float exact_scale(uint32_t s, int j, int q) {
    return RUN ? block_scale(s, q) : block_scale(s, 2 * (j >> 1) + (q >> 1));
}

// kSteps consecutive 128-value steps of one 16-row tile in registers.
// FULL: the number of steps is a multiple of kSteps, and a row's scales are read
// four (two) steps at a time; else step by step, and steps past the last one
// read the last one again (their products are skipped).
// ODD (K % 128 != 0; MX formats): 16-byte chunks past K count as zero codes with
// scale 2^0, and scales are read byte by byte (their rows start at any byte).
// Loads are never under a branch: the compiler counts them to know which ones
// have arrived, and where two paths meet it waits for all.
template <int F, int kSteps, bool FULL, bool ODD>
struct Tile {
    static constexpr int kL = loads_per_step(F);
    u32x4 c[kSteps * kL];
    uint32_t s[F == kBf16 ? 1 : kSteps];     // 4 blocks' scales (ODD: this lane's alone)

    // first value of chunk l of step st for lane quarter q: 16 bytes are 32 E2M1
    // or 16 E4M3 values
    static __device__ __forceinline__ int64_t value(int st, int l, int q) {
        return (int64_t)st * 128 + (F == kFp4 ? q * 32 : l * 64 + q * 16);
    }

    // codes16(byte), scale16/8/4(byte), scale1(byte): loads of the row at a byte of
    // it, the lane's 16 q included for codes
    template <class Src>
    __device__ __forceinline__ void load(const Src& src, int step, int last, int64_t K, int q) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int st = ODD || !FULL ? min(step + i, last - 1) : step + i;
#pragma unroll
            for (int l = 0; l < kL; ++l) {
                // ODD: a chunk past K reads the row's first 16 bytes instead (the
                // lane's 16 q taken back: a row may have no more than those)
                const bool in = !ODD || value(st, l, q) < K;
                c[i * kL + l] =
                    src.codes16(in ? (uint32_t)(st * bytes_per_step(F)) : 0u, in ? l * 64 : -16 * q);
            }
        }
        if constexpr (F == kBf16) {
        } else if constexpr (ODD) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int st = min(step + i, last - 1);
                const bool in = (int64_t)st * 128 + q * 32 < K;
                s[i] = src.scale1(in ? (uint32_t)(st * 4 + q) : 0u);
            }
        } else if constexpr (FULL && kSteps % 4 == 0) {
#pragma unroll
            for (int i = 0; i < kSteps; i += 4) {
                const u32x4 v = src.scale16((uint32_t)(step + i) * 4);
                s[i] = v.x;
                s[i + 1] = v.y;
                s[i + 2] = v.z;
                s[i + 3] = v.w;
            }
        } else if constexpr (FULL && kSteps % 2 == 0) {
#pragma unroll
            for (int i = 0; i < kSteps; i += 2) {
                const auto v = src.scale8((uint32_t)(step + i) * 4);
                s[i] = v.x;
                s[i + 1] = v.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) s[i] = src.scale4((uint32_t)min(step + i, last - 1) * 4);
        }
    }
    // the operand of step i, and its scale: this lane's block in the low byte
    __device__ __forceinline__ void codes(u32x4 (&o)[kL], int i, int st, int64_t K, int q) const {
#pragma unroll
        for (int l = 0; l < kL; ++l) {
            o[l] = c[i * kL + l];
            if constexpr (ODD)
                if (!(value(st, l, q) < K)) o[l] = u32x4{0, 0, 0, 0};
        }
    }
    __device__ __forceinline__ uint32_t scale(int i, int st, int64_t K, int q) const {
        if constexpr (F == kBf16) return 0;
        else if constexpr (ODD) return (int64_t)st * 128 + q * 32 < K ? s[i] : 127u;
        else return s[i] >> (8 * q);
    }
};

// Loads of a weight tile: buffer descriptors of its 16 rows (no bytes where there
// is no tile to load: the loads return zeros and touch no memory), the lane's row
// as an offset.
struct WSrc {
    __amdgpu_buffer_rsrc_t c, s;
    uint32_t crow, srow;
    template <int F>
    static __device__ __forceinline__ WSrc of(const uint8_t* codes, const uint8_t* scales, int64_t K,
                                              bool live, int lane) {
        const int cb = (int)row_bytes(F, K), sb = F == kBf16 ? 0 : (int)(K / 32);
        return WSrc{__builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(codes), 0, live ? 16 * cb : 0, 0x20000),
                    __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(scales), 0, live ? 16 * sb : 0, 0x20000),
                    (uint32_t)((lane & 15) * cb + (lane >> 4) * 16), (uint32_t)((lane & 15) * sb)};
    }
    __device__ __forceinline__ u32x4 codes16(uint32_t at, int imm) const {
        return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(c, (int)crow + imm, (int)at, 0));
    }
    __device__ __forceinline__ u32x4 scale16(uint32_t at) const {
        return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(s, (int)srow, (int)at, 0));
    }
    __device__ __forceinline__ uint2 scale8(uint32_t at) const {
        return __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(s, (int)srow, (int)at, 0));
    }
    __device__ __forceinline__ uint32_t scale4(uint32_t at) const {
        return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(s, (int)srow, (int)at, 0);
    }
    __device__ __forceinline__ uint32_t scale1(uint32_t at) const {     // at differs by lane
        return (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(s, (int)(srow + at), 0, 0);
    }
};
// ODD chunks differ by lane: the byte of the row goes into the lane's offset
struct WSrcOdd : WSrc {
    __device__ __forceinline__ u32x4 codes16(uint32_t at, int imm) const {
        return __builtin_bit_cast(u32x4,
                                  __builtin_amdgcn_raw_buffer_load_b128(c, (int)(crow + at) + imm, 0, 0));
    }
};

// An activation row as a lane reads it: its 16 bytes of K = 0 and its scales.
struct XRow {
    const uint8_t* codes;
    const uint8_t* scales;
    __device__ __forceinline__ u32x4 codes16(uint32_t at, int imm) const {
        return *reinterpret_cast<const u32x4*>(codes + at + imm);
    }
    __device__ __forceinline__ u32x4 scale16(uint32_t at) const {
        return *reinterpret_cast<const u32x4_a4*>(scales + at);
    }
    __device__ __forceinline__ uint2 scale8(uint32_t at) const {
        const u32x2_a4 v = *reinterpret_cast<const u32x2_a4*>(scales + at);
        return make_uint2(v.x, v.y);
    }
    __device__ __forceinline__ uint32_t scale4(uint32_t at) const {
        return *reinterpret_cast<const uint32_t*>(scales + at);
    }
    __device__ __forceinline__ uint32_t scale1(uint32_t at) const { return scales[at]; }
};
// The same with 32 values in a row: a lane's two loads of a step are at 32 q and
// 32 q + 16 (MXFP8 rows beside MXFP4 weights, exact products).
struct XRowRun : XRow {
    __device__ __forceinline__ u32x4 codes16(uint32_t at, int imm) const {
        return XRow::codes16(at, imm / 4);
    }
};
template <int F>
__device__ __forceinline__ XRow x_row(const uint8_t* codes, const uint8_t* scales, int64_t row, int64_t K,
                                      int lane) {
    return XRow{codes + row * row_bytes(F, K) + (lane >> 4) * 16,
                F == kBf16 ? nullptr : scales + row * (K / 32)};
}
__device__ __forceinline__ XRowRun x_row_run(const uint8_t* codes, const uint8_t* scales, int64_t row, int64_t K,
                                             int lane) {
    return XRowRun{{codes + row * K + (lane >> 4) * 32, scales + row * (K / 32)}};
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

// Steps [s0, s1) of wave's share of `steps` steps among `waves`, in whole groups
// of kSteps where FULL.
template <int kSteps, bool FULL>
__device__ __forceinline__ void share(int steps, int wave, int waves, int& s0, int& s1) {
    constexpr int g = FULL ? kSteps : 1;
    const int n = steps / g;
    s0 = wave * n / waves * g;
    s1 = (wave + 1) * n / waves * g;
}

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
// EXACT: exact products of MX operands (XF MXFP8; MXFP4 weights: rows by x_row_run).
template <int WF, int XF, int RT, int NT, int kSteps, bool FULL, bool ODD, bool EXACT, class First, class Next,
          class XRowOf, class Ending, class Done>
__device__ __forceinline__ void stream(int64_t K, int lane, First first, Next next, XRowOf xrow,
                                       Ending ending, Done done) {
    using U = Unit<RT>;
    using TW = Tile<WF, kSteps, FULL, ODD>;
    using TX = Tile<XF, kSteps, FULL, ODD>;
    // registers: two groups of weights, the sums, and kFirst tiles of X, of the
    // 256 that two waves a SIMD have
    constexpr int kHeld = 2 * RT * kSteps * (4 * TW::kL + 1) + 4 * RT * NT, kX = kSteps * (4 * TX::kL + 1);
    constexpr int kFirst = (232 - kHeld) / kX >= NT ? NT : (232 - kHeld) / kX;
    static_assert(kFirst >= 1 && NT <= 4, "a group of weights and a tile of rows fit");
    struct Group {
        TW w[RT];
    };
    const int q = lane >> 4;
    v4f acc[RT][NT];
    auto clear = [&]() {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[t][n] = v4f{0.f, 0.f, 0.f, 0.f};
    };
    auto load = [&](Group& g, const U& u, int step, bool live) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const WSrc src = WSrc::of<WF>(u.wc[t], u.ws[t], K, live, lane);
            if constexpr (ODD) g.w[t].load(WSrcOdd{src}, step, u.s1, K, q);
            else g.w[t].load(src, step, u.s1, K, q);
        }
    };
    auto mac = [&](const Group& g, const TX& x, auto nc, const U& u, int step) {
        constexpr int n = decltype(nc)::value;
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            if (FULL || i == 0 || step + i < u.s1) {
                u32x4 xc[TX::kL];
                x.codes(xc, i, step + i, K, q);
                const uint32_t xs = x.scale(i, step + i, K, q);
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    u32x4 wc[TW::kL];
                    g.w[t].codes(wc, i, step + i, K, q);
                    acc[t][n] = mac_step<WF, XF>(acc[t][n], wc, g.w[t].scale(i, step + i, K, q), xc, xs);
                }
            }
    };
    TX xs[kFirst];
    auto load_x = [&](TX& x, const U& u, int n, int step) { x.load(xrow(u, n), step, u.s1, K, q); };
    // f(integral_constant<n>) for the tiles A <= n < B that have rows
    auto tiles = [&](auto ac, auto bc, const U& u, auto&& f) {
        auto one = [&](auto nc) {
            constexpr int n = decltype(nc)::value;
            if constexpr (n >= decltype(ac)::value && n < decltype(bc)::value) {
                if constexpr (n == 0) f(nc);
                else if (n * 16 < u.rows) f(nc);
            }
        };
        one(std::integral_constant<int, 0>{});
        one(std::integral_constant<int, 1>{});
        one(std::integral_constant<int, 2>{});
        one(std::integral_constant<int, 3>{});
    };
    constexpr std::integral_constant<int, 0> k0{};
    constexpr std::integral_constant<int, kFirst> kF{};
    constexpr std::integral_constant<int, NT> kN{};
    // mac for all tiles of rows, with exact products: each chunk of rows is converted
    // once for TG tiles of weights, each chunk of weights once, and only one
    // chunk's values live at a time.  (TG: half of the tiles where the registers
    // are full, the compiler would spill rows.)
    auto mac_exact = [&](const Group& g, const TX* x, const U& u, int step) {
        constexpr bool kRun = WF == kFp4;
        constexpr int TG = RT == 4 && NT == 4 && kSteps > 1 ? 2 : RT;
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            if (FULL || i == 0 || step + i < u.s1) {
#pragma unroll
                for (int h = 0; h < 4 * (RT / TG); ++h) {
                    const int j = h / (RT / TG), t0 = h % (RT / TG) * TG;
                    __builtin_amdgcn_sched_barrier(0);
                    bf16x8 w[TG];
#pragma unroll
                    for (int t = 0; t < TG; ++t)
                        w[t] = exact_chunk<WF>(g.w[t0 + t].c + i * TW::kL,
                                                           exact_scale<kRun>(g.w[t0 + t].s[i], j, q), j);
                    tiles(k0, kN, u, [&](auto nc) {
                        constexpr int n = decltype(nc)::value;
                        const bf16x8 xv = exact_chunk<XF>(
                            x[n].c + i * TX::kL, exact_scale<kRun>(x[n].s[i], j, q), j);
#pragma unroll
                        for (int t = 0; t < TG; ++t)
                            acc[t0 + t][n] =
                                __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[t], xv, acc[t0 + t][n], 0, 0, 0);
                    });
                }
            }
    };
    U u;
    if (!first(u)) return;
    int step = u.s0;
    Group a, b;
    clear();
    load(a, u, step, true);
    // One turn: the next group's loads (of no bytes after the last one), then this
    // one's products.  Two turns make a round, the second one without work where
    // the groups are odd in number: a way out between them would give the compiler
    // a path from a turn to itself, on which it would wait for the loads in flight.
    bool live = true;
    auto turn = [&](Group& mine, Group& other) {
        U v = u;
        int vstep = step + kSteps;
        bool more = live;
        if (live && vstep >= u.s1) {
            more = next(v);
            vstep = v.s0;
            ending(u);
        }
        if (live)
            tiles(k0, kF, u, [&](auto nc) { load_x(xs[decltype(nc)::value], u, decltype(nc)::value, step); });
        __builtin_amdgcn_sched_barrier(0);       // loads in this order, products after them
        load(other, v, vstep, more);
        __builtin_amdgcn_sched_barrier(0);
        if (live) {
            if constexpr (EXACT) {
                static_assert(!EXACT || (kFirst == NT && XF == kFp8 && WF != kBf16 && !ODD), "all tiles in registers");
                mac_exact(mine, xs, u, step);
            } else {
                tiles(k0, kF, u, [&](auto nc) { mac(mine, xs[decltype(nc)::value], nc, u, step); });
                tiles(kF, kN, u, [&](auto nc) {
                    TX x;
                    load_x(x, u, decltype(nc)::value, step);
                    mac(mine, x, nc, u, step);
                });
            }
            if (step + kSteps >= u.s1) {
                done(acc, u);
                clear();
            }
        }
        u = v;
        step = vstep;
        live = __builtin_amdgcn_readfirstlane((int)more);
    };
    do {
        turn(a, b);
        turn(b, a);
    } while (live);
}

}  // namespace few
}  // namespace mx
