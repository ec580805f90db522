// Device helpers shared by the tile GEMM kernels (gfx950): raw buffer
// descriptors, direct global -> LDS loads, LDS-only barriers, wave-uniform
// values, and the bf16 store of a wave's 128 x 128 accumulators.
#pragma once
#include <utility>

#include "internal.h"
#include "mx_device.h"

namespace mx {
namespace {

constexpr uint32_t kRsrcWord3 = 0x00020000u;   // raw buffer, dword format

typedef int v4i __attribute__((ext_vector_type(4)));

// Raw buffer resource (no stride, dword format): base address, byte range
// (accesses at or past it read as zero).
__device__ __forceinline__ v4i make_rsrc(const void* p, int64_t bytes) {
    const int32_t n = bytes > 0x7fffffff ? 0x7fffffff : (int32_t)(bytes < 0 ? 0 : bytes);
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    return v4i{(int)(uint32_t)a, (int)((uint32_t)(a >> 32) & 0xffffu), n, (int)kRsrcWord3};
}

// LDS byte address of a __shared__ location.
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// Global -> LDS load of 16 (or 4) bytes per lane: lane l's bytes land at LDS
// address lds + OFF + 16*l (4*l).  Issued through inline asm so that the
// compiler does not track it: the kernel waits for these loads itself with
// vmcnt.  M0 carries the LDS address (declared clobbered: no other
// instruction in these kernels reads M0); one wait state separates the M0
// write from the load.  OFF, a constant, is added into M0 by the same scalar
// instruction that writes it, so that the loads of one stage share one base
// register instead of each keeping its own address live in a scalar register.
template <uint32_t OFF = 0>
__device__ __forceinline__ void dma_b128(const v4i& rsrc, uint32_t lds, uint32_t voff,
                                         uint32_t soff) {
    if constexpr (OFF == 0)
        asm volatile(
            "s_mov_b32 m0, %0\n\t"
            "s_nop 0\n\t"
            "buffer_load_dwordx4 %1, %2, %3 offen lds"
            :
            : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
            : "memory", "m0");
    else
        asm volatile(
            "s_add_u32 m0, %0, %4\n\t"
            "s_nop 0\n\t"
            "buffer_load_dwordx4 %1, %2, %3 offen lds"
            :
            : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff), "n"(OFF)
            : "memory", "m0", "scc");
}
template <uint32_t OFF = 0>
__device__ __forceinline__ void dma_b32(const v4i& rsrc, uint32_t lds, uint32_t voff,
                                        uint32_t soff) {
    if constexpr (OFF == 0)
        asm volatile(
            "s_mov_b32 m0, %0\n\t"
            "s_nop 0\n\t"
            "buffer_load_dword %1, %2, %3 offen lds"
            :
            : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
            : "memory", "m0");
    else
        asm volatile(
            "s_add_u32 m0, %0, %4\n\t"
            "s_nop 0\n\t"
            "buffer_load_dword %1, %2, %3 offen lds"
            :
            : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff), "n"(OFF)
            : "memory", "m0", "scc");
}

// Compile-time loop: f(integral_constant<int, 0>) ... f(integral_constant<int, N-1>),
// so that register arrays are only ever indexed by constants.
template <class Fn, int... I>
__device__ __forceinline__ void static_for_impl(Fn&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class Fn>
__device__ __forceinline__ void static_for(Fn&& f) {
    static_for_impl(f, std::make_integer_sequence<int, N>{});
}

// Workgroup barrier after this wave's LDS reads and writes have completed;
// global loads and stores still in flight (including loads into LDS, which
// the caller waits for with vmcnt) are not waited for.  The memory clobber
// keeps the compiler from moving LDS accesses across it.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Tile coordinates are wave-uniform but come from LDS reads; moving them to
// scalar registers keeps buffer descriptors and LDS-DMA addresses scalar.
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uni64(int64_t v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// The lane index, computed where it is used: a volatile computation is not
// hoisted, so no per-lane value has to stay live across the tile loops (where
// it would take a register, or a scratch slot whose reload waits with vmcnt
// for every store and load in flight).
__device__ __forceinline__ int lane_now() {
    int l;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
    return l;
}

__device__ __forceinline__ uint2 pack4_bf16(const float (&v)[4]) {
    return make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
}

// The plain epilogue straight from the registers, for tiles whose LDS holds
// the next tile's operands.  After the same v_permlane16_swap pairing, lane
// (r16, q) holds 8 consecutive columns of row i*16 + r16 for each jp: with
// jp = 2c and 2c + 1, the four lanes of a row hold the eight 16-byte chunks
// of 128-byte line c of the wave's row.  One DPP rotation by 8 within each
// 16-lane row then hands lane r16 < 8 the jp = 2c chunk of row r16 + 8, and
// lane r16 >= 8 the jp = 2c + 1 chunk of row r16 - 8, so that each store
// instruction writes whole lines: rows (r16 & 7) of the block, then rows 8
// + (r16 & 7), with lanes r16 < 8 on the jp = 2c half of the line and lanes
// r16 >= 8 on the other.  (Stored as the pairs left the swap, each
// instruction would write half lines, and the output would cost more.)
// gs: the tile's per-group output scale; rs: the wave's 128 routing weights
// in LDS (rows wm*128 ..), or null.  Nothing here reads global memory: a
// global load would wait (vmcnt) for every store and load in flight.
// part (a chunk of a split tail tile): the fp32 accumulators go instead, as
// they are, to the wave's blocks of a partial tile there (block (i, j) at
// byte (i * 8 + j) * 1024, lane l's 16 bytes at 16 l).  Both outputs share
// one pass over the row blocks, so the accumulators are read one way only.
// SCALED: the accumulators are multiplied by gs (and the row's rs) before
// the conversion; otherwise gs and rs are not read (the kernel variant for
// launches without output scales).
template <bool SCALED>
__device__ __forceinline__ void store_tile_bf16_regs(v4f (&acc)[8][8], const GemmProblem& p,
                                                     int g, int64_t m0, int64_t mvalid, int64_t n0,
                                                     int wm, int wn, int lane, float gs,
                                                     const float* rs, uint8_t* part = nullptr) {
    const int r16 = lane & 15, q = lane >> 4;
    const bool lo8 = r16 < 8;
    const int64_t rwave = m0 + wm * 128;
    const int rows_valid_w = (int)min((int64_t)128, max((int64_t)0, mvalid - wm * 128));
    uint16_t* C = reinterpret_cast<uint16_t*>(p.C) + (p.kgroup ? (int64_t)g * p.c_gstride : 0);
    const int64_t cw = n0 + wn * 128;
    // addresses: a wave-uniform base plus one 32-bit per-lane byte offset (the
    // lane's row r16 & 7 and its 16-byte chunk of line 0); rows, the second
    // half of a block and further lines only move the uniform base
    uint8_t* const Cw = reinterpret_cast<uint8_t*>(C + rwave * p.ldc + cw);
    const uint32_t ldb = (uint32_t)p.ldc * 2u;
    const int chunk0 = (lo8 ? 0 : 4) + 2 * (q & 1) + (q >> 1);
    const uint32_t loff = (uint32_t)(r16 & 7) * ldb + (uint32_t)chunk0 * 16u;
    // The rotation by 8 lanes of the rows' second halves, written only where
    // it lands: into the lanes r16 >= 8 (banks 2, 3) of s1, which start as
    // d0, and into the lanes r16 < 8 (banks 0, 1) of s2, which start as d1:
    // s1 = lo8 ? d0 : d1 of lane r16 ^ 8, s2 = lo8 ? d0 of lane r16 ^ 8 : d1.
    auto into_hi = [](uint32_t old, uint32_t v) {
        return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, 0x128, 0xf, 0xc, false);
    };
    auto into_lo = [](uint32_t old, uint32_t v) {
        return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, 0x128, 0xf, 0x3, false);
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // the accumulators live in AGPRs: pinned there at each row block, the
        // block moves to VGPRs only when it is converted (else the compiler
        // may move the whole tile up front and spill)
#pragma unroll
        for (int j = 0; j < 8; ++j) asm volatile("" : "+a"(acc[i][j]));
        if (part) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                *reinterpret_cast<v4f*>(part + (int64_t)(i * 8 + j) * 1024 + (uint32_t)lane * 16u) =
                    acc[i][j];
            __builtin_amdgcn_sched_barrier(0);
            continue;
        }
        const float sc = SCALED ? (rs ? rs[i * 16 + r16] * gs : gs) : 1.0f;
        const int rl1 = i * 16 + (r16 & 7), rl2 = rl1 + 8;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t d[2][4];                       // jp = 2c + h, after the swap
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int jp = 2 * c + h;
                float va[4], vb[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    va[v] = SCALED ? acc[i][2 * jp][v] * sc : acc[i][2 * jp][v];
                    vb[v] = SCALED ? acc[i][2 * jp + 1][v] * sc : acc[i][2 * jp + 1][v];
                }
                const uint2 a = pack4_bf16(va), b = pack4_bf16(vb);
                const auto x = __builtin_amdgcn_permlane16_swap(a.x, b.x, false, false);
                const auto y = __builtin_amdgcn_permlane16_swap(a.y, b.y, false, false);
                d[h][0] = x[0];
                d[h][1] = y[0];
                d[h][2] = x[1];
                d[h][3] = y[1];
            }
            uint32_t s1[4], s2[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                s1[v] = into_hi(d[0][v], d[1][v]);
                s2[v] = into_lo(d[1][v], d[0][v]);
            }
            const int chunk = chunk0 + 8 * c;
            if (cw + chunk * 8 < p.N) {
                uint8_t* const b1 = Cw + (int64_t)(i * 16) * ldb + c * 128;
                if (rl1 < rows_valid_w)
                    store_nt(b1 + loff, make_uint4(s1[0], s1[1], s1[2], s1[3]));
                if (rl2 < rows_valid_w)
                    store_nt(b1 + (int64_t)8 * ldb + loff, make_uint4(s2[0], s2[1], s2[2], s2[3]));
            }
        }
        // one row block at a time: the scheduler would otherwise read ahead
        // the accumulators of later blocks into registers the kernel has not
        // got (and spill them, the reload then waiting for every store)
        __builtin_amdgcn_sched_barrier(0);
    }
}

}  // namespace
}  // namespace mx
