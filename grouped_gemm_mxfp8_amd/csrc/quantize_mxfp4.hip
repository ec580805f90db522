// MXFP4 quantizer and its inverse (gfx950).
//
// A block of 32 values shares one E8M0 scale 2^X, X = floor(log2(amax)) - 2
// (2: the exponent of the largest E2M1 value, 6), and each element is the
// E2M1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) nearest to
// v * 2^-X, the even code of two equally near ones, saturated at 6.  X is
// bounded below by -127 (an all-zero block gets scale code 0); a block that
// holds an infinity or a NaN gets the NaN scale 255 and codes 0, so that what
// it stands for, and every product with it, is NaN.  Two codes share a byte,
// the even element in the low half.
//
// gfx950 converts a pair of bf16 values to two E2M1 codes with the division
// by the block scale in one instruction (v_cvt_scalef32_pk_fp4_bf16); equal,
// code for code, to the rule above on every finite bf16 pattern and every
// scale from 2^-127 to 2^125 (checked on the device).  So the row kernel has
// about 2 VALU instructions a value and is bound by HBM: 2 bytes read and
// 17/32 written a value.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "mx_device.h"

namespace mx {
namespace {

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));

// x is read once: loads that do not keep its lines in the caches leave those to
// the codes.  64 x (2048 x 1408) by columns 116 -> 96 us (4.9 TB/s), 16384 x 4096 by
// rows 32 -> 26.5 us (6.4 TB/s), inputs changing from call to call.
__device__ __forceinline__ uint4 load_once(const void* p) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
}

// elementwise max of two pairs of 16-bit magnitudes
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const u16x2 r = __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b));
    return __builtin_bit_cast(uint32_t, r);
}

// E8M0 code of a block from its amax as bf16 magnitude bits
__device__ __forceinline__ uint32_t e2m1_scale_code(uint32_t amax) {
    const uint32_t e = amax >> 7;
    return e == 255u ? 255u : e < 2u ? 0u : e - 2u;
}

// E2M1 codes of the eight bf16 values in p[0..3], in order
__device__ __forceinline__ uint32_t e2m1x8(const uint32_t (&p)[4], uint32_t code) {
    const float s = scale_from_code(code);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2v, p[0]), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2v, p[1]), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2v, p[2]), s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2v, p[3]), s, 3);
    return code == 255u ? 0u : w;
}

constexpr int kUnits = 4;   // 8-value units per lane in the flat kernels

// Rows are whole blocks, so the tensor is one flat run of blocks: four lanes
// share a block (8 values, one 16-byte load each) and find its amax with two
// DPP moves inside their quad.  A wave reads 1 KiB and writes 256 bytes of
// codes and 16 of scales an instruction.
__global__ void __launch_bounds__(256)
quant4_rows_kernel(const uint4* __restrict__ x, int64_t units, uint32_t* __restrict__ codes,
                   uint8_t* __restrict__ scales) {
    const int64_t u0 = (int64_t)blockIdx.x * (256 * kUnits) + threadIdx.x;
    uint4 v[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int64_t u = u0 + i * 256;
        if (u < units) v[i] = load_once(x + u);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int64_t u = u0 + i * 256;
        if (u >= units) break;              // whole quads: units % 4 == 0
        const uint32_t p[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t m = max2(max2(p[0] & 0x7fff7fffu, p[1] & 0x7fff7fffu),
                          max2(p[2] & 0x7fff7fffu, p[3] & 0x7fff7fffu));
        m = max2(m, m >> 16) & 0xffffu;
        m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, false));
        m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, false));
        const uint32_t c = e2m1_scale_code(m);
        codes[u] = e2m1x8(p, c);
        if ((threadIdx.x & 3) == 0) scales[u >> 2] = (uint8_t)c;
    }
}

// Columnwise copy: codes [C][R/2] of x [R][C], blocks along R.  One workgroup
// takes 256 rows x 64 columns through LDS; a thread then holds 32 rows of two
// neighbouring columns (32 dwords, one amax instruction for both), regroups
// them into row pairs and writes 16 bytes of each column.  Eight consecutive
// lanes hold the eight row blocks of a column pair, so a column's 128 bytes of
// codes leave as one line; each row block is skewed by 8 dwords in LDS, which
// puts the 8 x 8 lanes of a wave on 64 banks.
constexpr int kColRows = 256, kColCols = 64;
__global__ void __launch_bounds__(256)
quant4_cols_kernel(const uint16_t* __restrict__ x, int64_t R, int64_t C, uint8_t* __restrict__ codes,
                   uint8_t* __restrict__ scales) {
    __shared__ uint32_t tile[kColRows * (kColCols / 2) + 8 * (kColRows / 32)];
    const int64_t r0 = (int64_t)blockIdx.x * kColRows, c0 = (int64_t)blockIdx.y * kColCols;
    const int64_t bz = blockIdx.z;
    const uint16_t* xb = x + bz * R * C;
    const int tid = threadIdx.x;
    const int lc = (tid & 7) * 8;                       // first of 8 columns
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = i * 32 + (tid >> 3);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r0 + row < R && c0 + lc < C)
            v = load_once(xb + (r0 + row) * C + c0 + lc);
        *reinterpret_cast<uint4*>(&tile[row * 32 + i * 8 + lc / 2]) = v;
    }
    __syncthreads();
    const int rb = tid & 7, cp = tid >> 3;              // row block, column pair
    if (r0 + rb * 32 >= R || c0 + 2 * cp >= C) return;
    uint32_t d[32];
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
        d[r] = tile[(rb * 32 + r) * 32 + rb * 8 + cp];
        m = max2(m, d[r] & 0x7fff7fffu);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t c = e2m1_scale_code(h ? m >> 16 : m & 0xffffu);
        const uint32_t sel = h ? 0x07060302u : 0x05040100u;
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                p[j] = __builtin_amdgcn_perm(d[q * 8 + 2 * j + 1], d[q * 8 + 2 * j], sel);
            w[q] = e2m1x8(p, c);
        }
        const int64_t col = bz * C + c0 + 2 * cp + h;
        const int64_t blk = r0 / 32 + rb;
        *reinterpret_cast<uint4*>(codes + col * (R / 2) + blk * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        scales[col * (R / 32) + blk] = (uint8_t)c;
    }
}

// bf16 values of codes and scales: a lane expands 8 codes (one dword) to 16
// bytes.  Every value is exact (at most 2 significant bits, exponents down to
// 2^-128, which bf16 holds as a subnormal).
__global__ void __launch_bounds__(256)
dequant4_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t units,
                uint4* __restrict__ y) {
    const int64_t u0 = (int64_t)blockIdx.x * (256 * kUnits) + threadIdx.x;
    uint32_t w[kUnits], c[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int64_t u = u0 + i * 256;
        if (u < units) {
            w[i] = codes[u];
            c[i] = scales[u >> 2];
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int64_t u = u0 + i * 256;
        if (u >= units) break;
        const float s = scale_from_code(c[i]);
        uint4 o;
        o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 0));
        o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 1));
        o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 2));
        o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 3));
        if (c[i] == 255u) o = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
        y[u] = o;
    }
}

unsigned flat_grid(int64_t units) { return (unsigned)((units + 256 * kUnits - 1) / (256 * kUnits)); }

}  // namespace

hipError_t launch_quant4_rows(const uint16_t* x, int64_t n, uint8_t* codes, uint8_t* scales,
                              hipStream_t s) {
    hipLaunchKernelGGL(quant4_rows_kernel, dim3(flat_grid(n / 8)), dim3(256), 0, s,
                       reinterpret_cast<const uint4*>(x), n / 8, reinterpret_cast<uint32_t*>(codes),
                       scales);
    return hipGetLastError();
}

hipError_t launch_quant4_cols(const uint16_t* x, int64_t batch, int64_t R, int64_t C, uint8_t* codes,
                              uint8_t* scales, hipStream_t s) {
    const dim3 grid((unsigned)((R + kColRows - 1) / kColRows), (unsigned)((C + kColCols - 1) / kColCols),
                    (unsigned)batch);
    hipLaunchKernelGGL(quant4_cols_kernel, grid, dim3(256), 0, s, x, R, C, codes, scales);
    return hipGetLastError();
}

hipError_t launch_dequant4(const uint8_t* codes, const uint8_t* scales, int64_t n, uint16_t* y,
                           hipStream_t s) {
    hipLaunchKernelGGL(dequant4_kernel, dim3(flat_grid(n / 8)), dim3(256), 0, s,
                       reinterpret_cast<const uint32_t*>(codes), scales, n / 8,
                       reinterpret_cast<uint4*>(y));
    return hipGetLastError();
}

}  // namespace mx
