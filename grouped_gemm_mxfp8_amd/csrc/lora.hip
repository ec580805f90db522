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
// tiles most blocks of rows have one adapter whatever the batch's order.
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

__device__ __forceinline__ float dot8f(const float (&h)[8], const uint4& b, float s) {
    const uint32_t y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s += h[2 * i] * bf16_to_f32(y[i] & 0xffffu);
        s += h[2 * i + 1] * __uint_as_float(y[i] & 0xffff0000u);
    }
    return s;
}

template <bool FINE>
__global__ void __launch_bounds__(64 * DOWN_WAVES)
lora_down_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K, const uint16_t* __restrict__ a,
                 const int32_t* __restrict__ ids, const int32_t* __restrict__ order, const float* __restrict__ scale, int L, int r,
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

    // (sorted rows always go to the MFMA: a row's sums are then the same whatever rows are
    // beside it, and with them the same for any order among an adapter's rows)
    if (kinds > 2 && !order) {
        if (!FINE && blockIdx.z) return;
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
    const int64_t in = row < M ? row : M - 1;
    const uint16_t* const xr = x + (order ? order[in] : in) * K;
    // K in steps of 64, two MFMAs; a load takes 64 consecutive bytes of each row.  The last
    // step may have 32 values: its second load takes the last ones again, as zeros
    const int nk = (int)((K + 63) / 64);
    const int k_beg = nk * wave / DOWN_WAVES, k_end = nk * (wave + 1) / DOWN_WAVES;
    const bool rank_there = rank0 + r16 < r;
    for (int turn = 0; left; ++turn) {
        const int one = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        if (!FINE && (turn & 1) != (int)blockIdx.z) {        // grid.z: even and odd ones
            left &= ~__ballot(id == one);
            continue;
        }
        const uint16_t* const ar = a + ((int64_t)one * r + (rank_there ? rank0 + r16 : 0)) * K;
        v4f acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        auto steps = [&](auto nc, int ks) {       // n steps, their loads in flight together
            constexpr int n = decltype(nc)::value;
            uint4 xv[n][2], av[n][2];
#pragma unroll
            for (int i = 0; i < n; ++i) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int64_t k = min((int64_t)(ks + i) * 64 + u * 32, K - 32) + q * 8;
                    xv[i][u] = *reinterpret_cast<const uint4*>(xr + k);
                    av[i][u] = *reinterpret_cast<const uint4*>(ar + k);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < n; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint4 xz = xv[i][u], az = av[i][u];
                    if ((int64_t)(ks + i) * 64 + u * 32 >= K) xz = az = make_uint4(0, 0, 0, 0);
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

// ---- rows by adapter -----------------------------------------------------------------
// A counting sort in one workgroup.  The order among an adapter's rows is that of LDS
// atomics, any: no row's result depends on the rows beside it.
constexpr int SORT_THREADS = 1024, kSortMaxL = 8192;

__global__ void __launch_bounds__(SORT_THREADS)
lora_sort_kernel(const int32_t* __restrict__ ids, int M, int L, int32_t* __restrict__ order,
                 int32_t* __restrict__ sorted_ids) {
    __shared__ int s_at[kSortMaxL + 1];           // rows of each adapter, then where the next one goes
    __shared__ int s_wave[SORT_THREADS / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int l = tid; l <= L; l += SORT_THREADS) s_at[l] = 0;
    __syncthreads();
    // one atomic a wave where its rows have one adapter, as in a prompt; returns each
    // row's place among the counter's
    auto take = [&](int m, int key) -> int {
        const uint64_t here = __ballot(m < M);
        const int one = __builtin_amdgcn_readfirstlane(key);
        if (__ballot(m < M && key == one) == here) {
            int base = 0;
            if (lane == 0) base = atomicAdd(&s_at[one], (int)__popcll(here));
            return __builtin_amdgcn_readfirstlane(base) + lane;
        }
        return m < M ? atomicAdd(&s_at[key], 1) : 0;
    };
    auto key_of = [&](int m) {                    // rows without an adapter last
        const int id = m < M ? ids[m] : -1;
        return id >= 0 && id < L ? id : L;
    };
    // eight turns' ids in flight together
    for (int m0 = wave * 64; m0 < M; m0 += 8 * SORT_THREADS) {
        int key[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) key[i] = key_of(m0 + i * SORT_THREADS + lane);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (m0 + i * SORT_THREADS < M) take(m0 + i * SORT_THREADS + lane, key[i]);
    }
    __syncthreads();
    // exclusive prefix sums: a thread sums its run of counters, then the threads' sums
    const int run = (L + SORT_THREADS) / SORT_THREADS, beg = tid * run, end = min(beg + run, L + 1);
    int sum = 0;
    for (int l = beg; l < end; ++l) sum += s_at[l];
    const int incl = wave_prefix(sum, lane);
    if (lane == 63) s_wave[wave] = incl;
    __syncthreads();
    int at = incl - sum;
    for (int w = 0; w < wave; ++w) at += s_wave[w];
    for (int l = beg; l < end; ++l) {
        const int n = s_at[l];
        s_at[l] = at;
        at += n;
    }
    __syncthreads();
    for (int m0 = wave * 64; m0 < M; m0 += 8 * SORT_THREADS) {
        int key[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) key[i] = key_of(m0 + i * SORT_THREADS + lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int m = m0 + i * SORT_THREADS + lane;
            if (m - lane >= M) continue;
            const int to = take(m, key[i]);
            if (m < M) {
                order[to] = m;
                sorted_ids[to] = key[i] < L ? key[i] : -1;
            }
        }
    }
}

// ---- the layer for a few rows ----------------------------------------------------------
// y = x w^T + h b^T for up to 16 rows: reading w is what takes time.  A workgroup owns
// 16 CT columns; eight waves share K, each lane reading 32 consecutive bytes of its rows
// of w straight into the MFMA's registers.  Every workgroup reads all of x from the L2,
// so wide layers take more columns a workgroup.
//
// FUSED, for M r up to kFusedRanks (one token with an adapter of rank 32, two of rank 16):
// eight more waves make h = s a x meanwhile, every workgroup for itself, which is no more
// than it reads of w and saves a launch that takes as long as the rest (M = 1, r = 16,
// 4096 x 4096: two launches of 7 us each, one of 10).  h b^T follows when all are done.
// Otherwise four more waves make h b^T meanwhile, a value a thread, from h in memory.
// One order of every sum.
constexpr int FEW_WAVES = 8, kFusedRanks = 32;
constexpr int few_threads(bool fused) { return 64 * FEW_WAVES + (fused ? 64 * FEW_WAVES : 256); }

template <int CT, bool FUSED>
__global__ void __launch_bounds__(few_threads(FUSED))
lora_few_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K, const uint16_t* __restrict__ w, int64_t N,
                LowRank lr, const uint16_t* __restrict__ a, const float* __restrict__ scale,
                uint16_t* __restrict__ y) {
    __shared__ v4f s_sum[FEW_WAVES][CT][64];
    __shared__ float s_h[FUSED ? kFusedRanks : 1];
    __shared__ v4f s_low[FUSED ? 1 : CT][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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
    } else if constexpr (!FUSED) {
        const int at = tid - 64 * FEW_WAVES, m = at >> 4, id = m < M ? lr.id[m] : -1, r = lr.r;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const int64_t n = n0 + c * 16 + (at & 15);
            float low = 0.f;
            if (id >= 0 && id < lr.L && n < N) {
                const uint16_t* const h = lr.h + m * (2 * r);
                const uint16_t* const b = lr.b + ((int64_t)id * N + n) * r;
#pragma unroll 4
                for (int k = 0; k < r; k += 8) {
                    const uint4 bv = *reinterpret_cast<const uint4*>(b + k);
                    low = dot8(*reinterpret_cast<const uint4*>(h + r + k), bv, low);
                    low = dot8(*reinterpret_cast<const uint4*>(h + k), bv, low);
                }
            }
            // where the thread of row m and these four columns looks for it
            reinterpret_cast<float*>(&s_low[c][(at & 15) / 4 * 16 + m])[at & 3] = low;
        }
    } else {
        // two (row, rank) pairs of the M r at a time
        const int pairs = (int)M * lr.r;
        for (int i = (wave - FEW_WAVES) * 2; i < pairs; i += 2 * FEW_WAVES) {     // (r % 8 == 0: one row)
            const int m = i / lr.r, rank = i - m * lr.r, id = lr.id[m];
            if (id < 0 || id >= lr.L) continue;
            const uint16_t* const xr = x + m * K;
            const uint16_t* const ar = a + ((int64_t)id * lr.r + rank) * K;
            float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
            for (int64_t k = lane * 8; k < K; k += 512) {
                const uint4 xv = *reinterpret_cast<const uint4*>(xr + k);
                s0 = dot8(xv, *reinterpret_cast<const uint4*>(ar + k), s0);
                s1 = dot8(xv, *reinterpret_cast<const uint4*>(ar + K + k), s1);
            }
#pragma unroll
            for (int d = 32; d; d >>= 1) {
                s0 += __shfl_xor(s0, d);
                s1 += __shfl_xor(s1, d);
            }
            if (lane == 0) {
                const float sc = scale ? scale[id] : 1.f;
                s_h[i] = s0 * sc;
                s_h[i + 1] = s1 * sc;
            }
        }
    }
    __syncthreads();
    // thread (c, m, q): columns 16 c + 4 q .. + 3 of row m
    if (tid < 64 * CT) {
        const int c = tid >> 6, m = r16;
        const int64_t n = n0 + c * 16 + 4 * q;
        if (m >= M || n >= N) return;
        v4f v = s_sum[0][c][lane];
#pragma unroll
        for (int i = 1; i < FEW_WAVES; ++i) v += s_sum[i][c][lane];
        float f[4] = {0.f, 0.f, 0.f, 0.f};
        if constexpr (FUSED) {
            const int id = lr.id[m], r = lr.r;
            if (id >= 0 && id < lr.L) {
                const uint16_t* const b = lr.b + ((int64_t)id * N + n) * r;
                for (int k = 0; k < r; k += 8) {
                    float hv[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) hv[i] = s_h[m * r + k + i];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        f[e] = dot8f(hv, *reinterpret_cast<const uint4*>(b + e * r + k), f[e]);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = s_low[c][lane][e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] += v[e];
        *reinterpret_cast<uint2*>(y + m * N + n) = pack4_bf16(f);
    }
}

}  // namespace

bool lora_fuses(int64_t M, int r) { return M * r <= kFusedRanks; }

hipError_t launch_lora_few(const uint16_t* x, int64_t M, int64_t K, const uint16_t* w, int64_t N, const LowRank& lr,
                           const uint16_t* a, const float* scale, uint16_t* y, hipStream_t s) {
    // 16 columns a workgroup while that takes no more than two a CU (K = 4096, 16 rows, us:
    // N = 4096 15.4, with 32 columns 18.8; N = 8192 24.3 and 20.2; N = 14336 39.8 and 35.7)
    const int ct = N < 8192 ? 1 : 2;
    const dim3 grid((unsigned)((N + 16 * ct - 1) / (16 * ct)));
    const bool fused = lora_fuses(M, lr.r);
    const dim3 block(few_threads(fused));
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, s, x, M, K, w, N, lr, a, scale, y); };
    if (fused) ct == 1 ? go(lora_few_kernel<1, true>) : go(lora_few_kernel<2, true>);
    else ct == 1 ? go(lora_few_kernel<1, false>) : go(lora_few_kernel<2, false>);
    return hipGetLastError();
}

// Where adapters have eight rows each on average; rows in 32-bit bytes.
bool lora_sorts(int64_t M, int64_t K, int L) {
    return M > 256 && M <= 65536 && L <= kSortMaxL && 8 * (int64_t)L <= M && M * K < ((int64_t)1 << 30);
}
hipError_t launch_lora_sort(const int32_t* ids, int64_t M, int L, int32_t* order, int32_t* sorted_ids,
                            hipStream_t s) {
    hipLaunchKernelGGL(lora_sort_kernel, dim3(1), dim3(SORT_THREADS), 0, s, ids, (int)M, L, order, sorted_ids);
    return hipGetLastError();
}

hipError_t launch_lora_down(const uint16_t* x, int64_t M, int64_t K, const uint16_t* a, const int32_t* id,
                            const int32_t* order, const float* scale, int L, int r, uint16_t* h, hipStream_t s) {
    if (M == 0) return hipSuccess;
    const unsigned blocks = (unsigned)((M + 15) / 16);
    const dim3 block(64 * DOWN_WAVES);
    if (!order && M * r <= 65536)          // 4096 workgroups, of which a prompt's blocks use one in sixteen
        hipLaunchKernelGGL(lora_down_kernel<true>, dim3(blocks, (unsigned)(r / 4), 4), block, 0, s, x, M, K, a, id,
                           order, scale, L, r, h);
    else
        hipLaunchKernelGGL(lora_down_kernel<false>, dim3(blocks, (unsigned)((r + 15) / 16), 2), block, 0, s, x, M, K, a,
                           id, order, scale, L, r, h);
    return hipGetLastError();
}

}  // namespace mx
