// The adapters' down projection (gfx950): h[m] = scale[l] x[m] a[l]^T with l the
// adapter of row m, stored as the high and the low bf16 part of each fp32 value (the
// sum of both is off by at most 2^-16 of it, so the product with b that follows
// loses nothing a bf16 result could show).
//
// One workgroup of eight waves per 16 rows and 16 ranks; the waves share K, each lane
// reading 32 consecutive bytes of its row.  The workgroup goes through the adapters
// that its rows have: one pass over x and a where all have the same, as in a prompt.
#include "bf16_tiles.h"

namespace mx {
namespace {

constexpr int DOWN_WAVES = 8;

__global__ void __launch_bounds__(64 * DOWN_WAVES)
lora_down_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K, const uint16_t* __restrict__ a,
                 const int32_t* __restrict__ ids, const float* __restrict__ scale, int L, int r,
                 uint16_t* __restrict__ h) {
    __shared__ v4f s_sum[DOWN_WAVES][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int r16 = lane & 15, q = lane >> 4;
    const int64_t row = (int64_t)blockIdx.x * 16 + r16;
    const int rank0 = blockIdx.y * 16;
    int id = row < M ? ids[row] : -1;
    if (id >= L) id = -1;
    const uint16_t* const xr = x + (row < M ? row : M - 1) * K;
    // K in steps of 64: 16 values a lane, two MFMAs; the last step may have 32
    const int nk = (int)((K + 63) / 64);
    const int k_beg = nk * wave / DOWN_WAVES, k_end = nk * (wave + 1) / DOWN_WAVES;
    const bool rank_there = rank0 + r16 < r;
    uint64_t left = __ballot(id >= 0);
    while (left) {
        const int one = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint16_t* const ar = a + ((int64_t)one * r + (rank_there ? rank0 + r16 : 0)) * K;
        v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int ks = k_beg; ks < k_end; ++ks) {
            const int64_t k = (int64_t)ks * 64 + q * 16;
            uint4 xv[2] = {}, av[2] = {};
            if (k < K) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    xv[u] = *reinterpret_cast<const uint4*>(xr + k + 8 * u);
                    av[u] = *reinterpret_cast<const uint4*>(ar + k + 8 * u);
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av[u]),
                                                              __builtin_bit_cast(bf16x8, xv[u]), acc, 0, 0, 0);
        }
        // lane (r16, q): row r16, ranks 4 q .. + 3
        s_sum[wave][lane] = acc;
        __syncthreads();
        if (wave == 0 && id == one) {
            v4f v = s_sum[0][lane];
#pragma unroll
            for (int w = 1; w < DOWN_WAVES; ++w) v += s_sum[w][lane];
            const float sc = scale ? scale[one] : 1.f;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float f = v[e] * sc;
                hi[e] = f32_to_bf16(f);
                const float rest = f - bf16_to_f32(hi[e]);
                // (an infinity has no rest: inf - inf would make it a NaN)
                lo[e] = __builtin_isfinite(rest) ? f32_to_bf16(rest) : 0u;
            }
            const int rank = rank0 + 4 * q;
            if (rank < r) {
                uint16_t* const at = h + row * (2 * r) + rank;
                *reinterpret_cast<uint2*>(at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
                *reinterpret_cast<uint2*>(at + r) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
            }
        }
        __syncthreads();
        left &= ~__ballot(id == one);
    }
}

}  // namespace

hipError_t launch_lora_down(const uint16_t* x, int64_t M, int64_t K, const uint16_t* a, const int32_t* id,
                            const float* scale, int L, int r, uint16_t* h, hipStream_t s) {
    if (M == 0) return hipSuccess;
    const dim3 grid((unsigned)((M + 15) / 16), (unsigned)((r + 15) / 16));
    hipLaunchKernelGGL(lora_down_kernel, grid, dim3(64 * DOWN_WAVES), 0, s, x, M, K, a, id, scale, L, r, h);
    return hipGetLastError();
}

}  // namespace mx
