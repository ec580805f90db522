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
#include "bf16_tiles.h"

namespace mx {
namespace {

constexpr int DOWN_WAVES = 8;

// The two bf16 parts of f.  (An infinity has no rest: inf - inf would make it a NaN.)
__device__ __forceinline__ void split2(float f, uint32_t& hi, uint32_t& lo) {
    hi = f32_to_bf16(f);
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

template <bool FINE>
__global__ void __launch_bounds__(64 * DOWN_WAVES)
lora_down_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K, const uint16_t* __restrict__ a,
                 const int32_t* __restrict__ ids, const float* __restrict__ scale, int L, int r,
                 uint16_t* __restrict__ h) {
    __shared__ v4f s_sum[DOWN_WAVES][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int r16 = lane & 15, q = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * 16, row = row0 + r16;
    int id = row < M ? ids[row] : -1;
    if (id >= L) id = -1;
    const float sc = scale && id >= 0 ? scale[id] : 1.f;
    uint64_t left = __ballot(id >= 0);
    int kinds = 0;                                // adapters among the rows, up to three
    for (uint64_t m = left; m && kinds < 3; ++kinds)
        m &= ~__ballot(id == __builtin_amdgcn_readlane(id, __builtin_ctzll(m)));
    // (a row's scale and parts: what lane (r16, q) holds of its row's four ranks)
    auto store = [&](const v4f& v, float by, int64_t to, int rank) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2(v[e] * by, hi[e], lo[e]);
        uint16_t* const at = h + to * (2 * r) + rank;
        *reinterpret_cast<uint2*>(at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
        *reinterpret_cast<uint2*>(at + r) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
    };

    if (kinds > 2) {
        // FINE: grid.y counts ranks in fours, grid.z rows in fours; else both in sixteens
        const int rank_beg = blockIdx.y * (FINE ? 4 : 16), rank_end = min(r, rank_beg + (FINE ? 4 : 16));
        const int row_beg = FINE ? blockIdx.z * 4 : 0, row_end = FINE ? row_beg + 4 : 16;
        const int part = wave & 1;                // of K: 512 values in turn
        for (int rb = row_beg; rb < row_end; rb += 4) {
            const int mine = rb + (wave >> 1);
            const int own = __builtin_amdgcn_readlane(id, mine);
            const float by = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(sc), mine));
            const uint16_t* const xr = x + min(row0 + mine, M - 1) * K;
            for (int rank = rank_beg; rank < rank_end; rank += 4) {
                v4f s = {0.f, 0.f, 0.f, 0.f};
                if (own >= 0) {
                    const uint16_t* const ar = a + ((int64_t)own * r + rank) * K;
                    // twenty loads in flight: 4096 values of K in the two waves
                    for (int64_t k0 = part * 512 + lane * 8; k0 - lane * 8 < K; k0 += 4096) {
                        uint4 xv[4], av[4][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int64_t k = k0 + i * 1024, kc = k < K ? k : K - 8;
                            xv[i] = *reinterpret_cast<const uint4*>(xr + kc);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                av[i][e] = *reinterpret_cast<const uint4*>(ar + e * K + kc);
                        }
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (k0 + i * 1024 < K)
#pragma unroll
                                for (int e = 0; e < 4; ++e) s[e] = dot8(xv[i], av[i][e], s[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int d = 32; d; d >>= 1) s[e] += __shfl_xor(s[e], d);
                }
                if (lane == 0) s_sum[wave][0] = s;
                __syncthreads();
                if (own >= 0 && part == 0 && lane == 0) store(s_sum[wave][0] + s_sum[wave + 1][0], by, row0 + mine, rank);
                __syncthreads();
            }
        }
        return;
    }

    if (FINE && (blockIdx.y % 4 || blockIdx.z)) return;
    const int rank0 = blockIdx.y * (FINE ? 4 : 16);
    const uint16_t* const xr = x + (row < M ? row : M - 1) * K;
    // K in steps of 64: 16 values a lane, two MFMAs; the last step may have 32, whose
    // other lanes read the last values again and count them as zeros
    const int nk = (int)((K + 63) / 64);
    const int k_beg = nk * wave / DOWN_WAVES, k_end = nk * (wave + 1) / DOWN_WAVES;
    const bool rank_there = rank0 + r16 < r;
    while (left) {
        const int one = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint16_t* const ar = a + ((int64_t)one * r + (rank_there ? rank0 + r16 : 0)) * K;
        v4f acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        auto steps = [&](auto nc, int ks) {       // n steps, their loads in flight together
            constexpr int n = decltype(nc)::value;
            uint4 xv[n][2], av[n][2];
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const int64_t k = (int64_t)(ks + i) * 64 + q * 16, kc = k < K ? k : K - 16;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    xv[i][u] = *reinterpret_cast<const uint4*>(xr + kc + 8 * u);
                    av[i][u] = *reinterpret_cast<const uint4*>(ar + kc + 8 * u);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < n; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint4 xz = xv[i][u], az = av[i][u];
                    if ((int64_t)(ks + i) * 64 + q * 16 >= K) xz = az = make_uint4(0, 0, 0, 0);
                    acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, az),
                                                                     __builtin_bit_cast(bf16x8, xz), acc[u], 0, 0, 0);
                }
        };
        int ks = k_beg;
        for (; ks + 8 <= k_end; ks += 8) steps(std::integral_constant<int, 8>{}, ks);
        for (; ks + 2 <= k_end; ks += 2) steps(std::integral_constant<int, 2>{}, ks);
        if (ks < k_end) steps(std::integral_constant<int, 1>{}, ks);
        // lane (r16, q): row r16, ranks 4 q .. + 3
        s_sum[wave][lane] = acc[0] + acc[1];
        __syncthreads();
        if (wave == 0 && id == one && rank0 + 4 * q < r) {
            v4f v = s_sum[0][lane];
#pragma unroll
            for (int w = 1; w < DOWN_WAVES; ++w) v += s_sum[w][lane];
            store(v, sc, row, rank0 + 4 * q);
        }
        __syncthreads();
        left &= ~__ballot(id == one);
    }
}

// ---- the layer for a few rows ----------------------------------------------------------
// y = x w^T + h b^T for up to 16 rows: reading w is what takes time.  A workgroup owns
// 16 CT columns; eight waves share K, each lane reading 32 consecutive bytes of its rows
// of w straight into the MFMA's registers; four more waves make the adapters' part
// meanwhile, a value a thread.  Every workgroup reads all of x from the L2, so wide
// layers take more columns a workgroup.  One order of every sum.
constexpr int FEW_WAVES = 8;

template <int CT>
__global__ void __launch_bounds__(64 * FEW_WAVES + 256)
lora_few_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K, const uint16_t* __restrict__ w, int64_t N,
                LowRank lr, uint16_t* __restrict__ y) {
    __shared__ v4f s_sum[FEW_WAVES][CT][64];
    __shared__ float s_low[CT][16][16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int r16 = lane & 15, q = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * CT);
    if (wave < FEW_WAVES) {
        const uint16_t* wr[CT];
        // (columns past the layer read its last ones; they are not stored)
#pragma unroll
        for (int c = 0; c < CT; ++c) wr[c] = w + min(n0 + c * 16 + r16, N - 1) * K;
        const uint16_t* const xr = x + min((int64_t)r16, M - 1) * K;
        v4f acc[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[c] = v4f{0.f, 0.f, 0.f, 0.f};
        // the last step may have 32 values: the other lanes read the last ones again and
        // count them as zeros
        const int nk = (int)((K + 63) / 64);
        const int k_beg = nk * wave / FEW_WAVES, k_end = nk * (wave + 1) / FEW_WAVES;
#pragma unroll (CT == 1 ? 8 : 4)
        for (int ks = k_beg; ks < k_end; ++ks) {
            const int64_t k = (int64_t)ks * 64 + q * 16, kc = k < K ? k : K - 16;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint4 xv = *reinterpret_cast<const uint4*>(xr + kc + 8 * u);
                if (k >= K) xv = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    uint4 wv = *reinterpret_cast<const uint4*>(wr[c] + kc + 8 * u);
                    if (k >= K) wv = make_uint4(0, 0, 0, 0);
                    acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wv),
                                                                     __builtin_bit_cast(bf16x8, xv), acc[c], 0, 0, 0);
                }
            }
        }
        // lane (r16, q): row r16, columns 4 q .. + 3 of the sixteen
#pragma unroll
        for (int c = 0; c < CT; ++c) s_sum[wave][c][lane] = acc[c];
    } else {
        const int at = (int)threadIdx.x - 64 * FEW_WAVES, m = at >> 4;
        const int id = m < M ? lr.id[m] : -1;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const int64_t n = n0 + c * 16 + (at & 15);
            float low = 0.f;
            if (id >= 0 && id < lr.L && n < N) {
                const uint16_t* const h = lr.h + m * (2 * lr.r);
                const uint16_t* const b = lr.b + ((int64_t)id * N + n) * lr.r;
#pragma unroll 4
                for (int k = 0; k < lr.r; k += 8) {
                    const uint4 bv = *reinterpret_cast<const uint4*>(b + k);
                    low = dot8(*reinterpret_cast<const uint4*>(h + lr.r + k), bv, low);
                    low = dot8(*reinterpret_cast<const uint4*>(h + k), bv, low);
                }
            }
            s_low[c][m][at & 15] = low;
        }
    }
    __syncthreads();
    if (wave < CT) {
        v4f v = s_sum[0][wave][lane];
#pragma unroll
        for (int i = 1; i < FEW_WAVES; ++i) v += s_sum[i][wave][lane];
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = v[e] + s_low[wave][r16][4 * q + e];
        const int64_t n = n0 + wave * 16 + 4 * q;
        if (r16 < M && n < N) *reinterpret_cast<uint2*>(y + r16 * N + n) = pack4_bf16(f);
    }
}

}  // namespace

hipError_t launch_lora_few(const uint16_t* x, int64_t M, int64_t K, const uint16_t* w, int64_t N, const LowRank& lr,
                           uint16_t* y, hipStream_t s) {
    const dim3 block(64 * FEW_WAVES + 256);
    // 16 columns a workgroup while that takes no more than two a CU (K = 4096, 16 rows, us:
    // N = 4096 15.4, with 32 columns 18.8; N = 8192 24.3 and 20.2; N = 14336 39.8 and 35.7)
    const int ct = N < 8192 ? 1 : 2;
    const dim3 grid((unsigned)((N + 16 * ct - 1) / (16 * ct)));
    if (ct == 1) hipLaunchKernelGGL(lora_few_kernel<1>, grid, block, 0, s, x, M, K, w, N, lr, y);
    else hipLaunchKernelGGL(lora_few_kernel<2>, grid, block, 0, s, x, M, K, w, N, lr, y);
    return hipGetLastError();
}

hipError_t launch_lora_down(const uint16_t* x, int64_t M, int64_t K, const uint16_t* a, const int32_t* id,
                            const float* scale, int L, int r, uint16_t* h, hipStream_t s) {
    if (M == 0) return hipSuccess;
    const unsigned blocks = (unsigned)((M + 15) / 16);
    const dim3 block(64 * DOWN_WAVES);
    if (M * r <= 65536)          // 4096 workgroups, of which a prompt's blocks use one in sixteen
        hipLaunchKernelGGL(lora_down_kernel<true>, dim3(blocks, (unsigned)(r / 4), 4), block, 0, s, x, M, K, a, id,
                           scale, L, r, h);
    else
        hipLaunchKernelGGL(lora_down_kernel<false>, dim3(blocks, (unsigned)((r + 15) / 16)), block, 0, s, x, M, K, a,
                           id, scale, L, r, h);
    return hipGetLastError();
}

}  // namespace mx
