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

// One operand's 16-row tile as a lane sees it: its own row (codes at the
// lane's 16 bytes of K = 0, scales at K = 0).
struct Row {
    const uint8_t* codes;
    const uint8_t* scales;
};
template <int F>
__device__ __forceinline__ Row row_of(const uint8_t* codes, const uint8_t* scales, int64_t row, int64_t K,
                                      int lane) {
    return Row{codes + row * row_bytes(F, K) + (lane >> 4) * 16,
               F == kBf16 ? nullptr : scales + row * (K / 32)};
}

// kSteps consecutive 128-value steps of one tile in registers.  Steps at or
// past `last` (uniform) repeat step last - 1 and are skipped by the caller:
// the loads stay in range without a branch per lane.
// ODD (K % 128 != 0; MX formats): 16-byte chunks past K read as zero codes,
// their scales as 2^0, and scales are read byte by byte (their rows start at
// any byte).
template <int F, int kSteps, bool ODD>
struct Tile {
    static constexpr int kL = loads_per_step(F);
    u32x4 c[kSteps * kL];
    uint32_t s[F == kBf16 ? 1 : kSteps];     // 4 blocks' scales (ODD: this lane's alone)

    __device__ __forceinline__ void load(const Row& r, int step, int last, int64_t K, int q) {
        if constexpr (ODD) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int st = min(step + i, last - 1);
#pragma unroll
                for (int l = 0; l < kL; ++l) {
                    // first value of the chunk: E2M1 16 bytes are 32 values, E4M3 16
                    const int64_t k0 = F == kFp4 ? (int64_t)st * 128 + q * 32 : (int64_t)st * 128 + l * 64 + q * 16;
                    c[i * kL + l] = u32x4{0, 0, 0, 0};
                    if (k0 < K)
                        c[i * kL + l] = *reinterpret_cast<const u32x4*>(
                            r.codes + (int64_t)st * bytes_per_step(F) + l * 64);
                }
                s[i] = 127;
                if ((int64_t)st * 128 + q * 32 < K) s[i] = r.scales[(int64_t)st * 4 + q];
            }
        } else {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int st = min(step + i, last - 1);
#pragma unroll
                for (int l = 0; l < kL; ++l)
                    c[i * kL + l] = *reinterpret_cast<const u32x4*>(
                        r.codes + (int64_t)st * bytes_per_step(F) + l * 64);
            }
            if constexpr (F != kBf16) {
                if (kSteps % 4 == 0 && step + kSteps <= last) {
#pragma unroll
                    for (int i = 0; i + 3 < kSteps; i += 4) {
                        const u32x4 v = *reinterpret_cast<const u32x4_a4*>(r.scales + (int64_t)(step + i) * 4);
                        s[i] = v.x;
                        s[i + 1] = v.y;
                        s[i + 2] = v.z;
                        s[i + 3] = v.w;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kSteps; ++i)
                        s[i] = *reinterpret_cast<const uint32_t*>(r.scales + (int64_t)min(step + i, last - 1) * 4);
                }
            }
        }
    }
    // the scale operand of step i: this lane's block in the low byte
    __device__ __forceinline__ uint32_t scale(int i, int q) const {
        if constexpr (F == kBf16) return 0;
        else if constexpr (ODD) return s[i];
        else return s[i] >> (8 * q);
    }
};

// acc[RT][NT] += W rows . X rows over the steps [s0, s1) (uniform), kSteps at
// a time with the next group's weights in flight.
template <int WF, int XF, int RT, int NT, int kSteps, bool ODD>
__device__ __forceinline__ void mac_rows(v4f (&acc)[RT][NT], const Row (&w)[RT], const Row (&x)[NT], int s0,
                                         int s1, int64_t K, int q) {
    if (s0 >= s1) return;
    using TW = Tile<WF, kSteps, ODD>;
    using TX = Tile<XF, 1, ODD>;
    auto compute = [&](const TW (&tw)[RT], int step) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if (i == 0 || step + i < s1) {
                TX tx[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) tx[n].load(x[n], step + i, s1, K, q);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int t = 0; t < RT; ++t)
                        acc[t][n] = mac_step<WF, XF>(acc[t][n], tw[t].c + i * TW::kL, tw[t].scale(i, q),
                                                     tx[n].c, tx[n].scale(0, q));
            }
        }
    };
    auto load = [&](TW (&tw)[RT], int step) {
#pragma unroll
        for (int t = 0; t < RT; ++t) tw[t].load(w[t], step, s1, K, q);
    };
    TW a[RT], b[RT];
    load(a, s0);
    for (int st = s0; st < s1; st += 2 * kSteps) {
        const bool more = st + kSteps < s1;
        if (more) load(b, st + kSteps);
        compute(a, st);
        if (more) {
            if (st + 2 * kSteps < s1) load(a, st + 2 * kSteps);
            compute(b, st + kSteps);
        }
    }
}

}  // namespace few
}  // namespace mx
