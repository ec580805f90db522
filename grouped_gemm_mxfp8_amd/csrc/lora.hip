// The adapter linear's kernels beside the tiles (gfx950): the adapters' down projection
// as a launch of its own, rows in the order of their adapters, and the whole layer for a
// few rows.
#include "lora_down.h"

namespace mx {
namespace {

constexpr int DOWN_WAVES = 8;

template <int RB, bool FINE>
__global__ void __launch_bounds__(64 * DOWN_WAVES)
lora_down_kernel(LoraDown p) {
    __shared__ v4f s_sum[DOWN_WAVES][RB][64];
    lora_down<DOWN_WAVES, RB, FINE>(p, (int)blockIdx.x, (int)blockIdx.y, (int)blockIdx.z, s_sum);
}

// ---- rows by adapter -----------------------------------------------------------------
// A counting sort in one workgroup.  The order among an adapter's rows is that of LDS
// atomics, any: sorted rows always take the MFMA, where no row's result depends on the rows
// beside it.
constexpr int SORT_THREADS = 1024, kSortMaxL = 8192;

__global__ void __launch_bounds__(SORT_THREADS)
lora_sort_kernel(const int32_t* __restrict__ ids, int M, int L, int32_t* __restrict__ order,
                 int32_t* __restrict__ sorted_ids, int64_t* __restrict__ offs) {
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
        offs[l] = at;
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

// h of rows with M r up to kFusedRanks, by eight waves: two (row, rank) pairs of the M r at a
// time.
__device__ __forceinline__ void few_h(const uint16_t* x, int64_t M, int64_t K, const LowRank& lr, const uint16_t* a,
                                      const float* scale, int wave, int lane, float* s_h) {
    const int pairs = (int)M * lr.r;
    for (int i = wave * 2; i < pairs; i += 2 * FEW_WAVES) {     // (r % 8 == 0: one row)
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
        few_h(x, M, K, lr, a, scale, wave - FEW_WAVES, lane, s_h);
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

// The same for wide layers.  One workgroup a CU takes sixteen columns after sixteen, and its
// eight waves read their shares of w as one stream over all of them, the next loads in flight
// before the current ones are used; x, which every sixteen columns need, stays in the LDS.
// The other waves make the adapters' part of the same columns meanwhile, add the eight sums
// to it and store, a value a thread.  K = 4096, us with the kernel above and here: 28672
// columns, 1 row, r = 16 57.6 and 44.5 (5.9 TB/s past a start of 5 us), 16 rows, r = 64 71 and
// 62; 14336 columns 31.3 and 27.3, 39.7 and 38.0.
constexpr int kWideX = 136 * 1024;
// Bytes between rows of x in the LDS: a column's sixteen on different banks.
__device__ __host__ constexpr int64_t wide_pitch(int64_t K) { return (K * 2 + 255) / 256 * 256 + 16; }

template <bool FUSED>
__global__ void __launch_bounds__(few_threads(FUSED))
lora_wide_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K, const uint16_t* __restrict__ w, int64_t N,
                 LowRank lr, const uint16_t* __restrict__ a, const float* __restrict__ scale,
                 uint16_t* __restrict__ y) {
    __shared__ __attribute__((aligned(16))) uint8_t s_x[kWideX];
    __shared__ v4f s_sum[2][FEW_WAVES][64];
    __shared__ float s_h[FUSED ? kFusedRanks : 1];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, q = lane >> 4;
    // whole rounds of sixteen columns a workgroup, and one of what is left, in even parts
    const int64_t round = (int64_t)gridDim.x * 16;
    const int whole = (int)(N / round);                                // at least one
    const int part = (int)((N - whole * round + gridDim.x - 1) / gridDim.x);
    const int64_t last_n = whole * round + (int64_t)blockIdx.x * part;
    const int last_width = (int)max((int64_t)0, min((int64_t)part, N - last_n));
    const int units = whole + (last_width > 0);
    auto first_of = [&](int u) { return u < whole ? u * round + (int64_t)blockIdx.x * 16 : last_n; };
    auto width_of = [&](int u) { return u < whole ? 16 : last_width; };
    const int pitch = (int)wide_pitch(K);
    auto stage_x = [&] {
        for (int m = 0; m < M; ++m)
            for (int c = tid; c < K / 8; c += few_threads(FUSED))
                *reinterpret_cast<uint4*>(s_x + m * pitch + c * 16) = *reinterpret_cast<const uint4*>(x + m * K + c * 8);
        __syncthreads();
    };

    // Every wave: one barrier for x, then one for each sixteen columns, behind which their sums
    // are read while the other half of s_sum is written.
    if (wave < FEW_WAVES) {
        constexpr int G = 4;                                // steps of 64 in K loaded together
        const int nk = (int)((K + 63) / 64);
        const int k_beg = nk * wave / FEW_WAVES, k_end = nk * (wave + 1) / FEW_WAVES;
        const int groups = (k_end - k_beg + G - 1) / G;     // (at least one: K >= 2048)
        const uint8_t* const xr = s_x + min((int64_t)r16, M - 1) * pitch;
        struct Group {
            uint4 w[G][2];
        };
        // a lane's place in a step.  The last step may have 32 values: the other lanes read
        // the last ones again and count them as zeros
        auto at = [&](int ks) { return (int64_t)ks * 64 + q * 16; };
        auto load = [&](Group& g, int unit, int group) {
            const uint16_t* const wr = w + (first_of(unit) + min(r16, width_of(unit) - 1)) * K;
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const int64_t k = at(k_beg + group * G + i), kc = k < K ? k : K - 16;
#pragma unroll
                for (int u = 0; u < 2; ++u) g.w[i][u] = *reinterpret_cast<const uint4*>(wr + kc + 8 * u);
            }
        };
        v4f acc = {0.f, 0.f, 0.f, 0.f};
        int unit = 0, group = 0;
        // uses the current group and loads the next one, if there is any
        auto turn = [&](const Group& cur, Group& nxt) {
            const bool ends = group + 1 == groups;
            const int nu = ends ? unit + 1 : unit, ng = ends ? 0 : group + 1;
            if (nu < units) load(nxt, nu, ng);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const int ks = k_beg + group * G + i;
                if (ks >= k_end) break;
                const int64_t k = at(ks), kc = k < K ? k : K - 16;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint4 wv = cur.w[i][u], xv = *reinterpret_cast<const uint4*>(xr + (kc + 8 * u) * 2);
                    if (k >= K) wv = xv = make_uint4(0, 0, 0, 0);
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wv),
                                                                  __builtin_bit_cast(bf16x8, xv), acc, 0, 0, 0);
                }
            }
            if (ends) {
                // lane (r16, q): row r16, columns 4 q .. + 3 of the sixteen
                s_sum[unit & 1][wave][lane] = acc;
                acc = v4f{0.f, 0.f, 0.f, 0.f};
                lds_barrier();
            }
            unit = nu;
            group = ng;
        };
        Group g0, g1;
        load(g0, 0, 0);
        stage_x();
        while (unit < units) {
            turn(g0, g1);
            if (unit < units) turn(g1, g0);
        }
        return;
    }

    stage_x();
    const int at = tid - 64 * FEW_WAVES, m = at >> 4, id = m < M ? lr.id[m] : -1, r = lr.r;
    const bool mine = id >= 0 && id < lr.L;
    if constexpr (FUSED) few_h(x, M, K, lr, a, scale, wave - FEW_WAVES, lane, s_h);
    for (int u = 0; u < units; ++u) {
        const int64_t n = first_of(u) + (at & 15);
        const bool there = m < M && (at & 15) < width_of(u), adapt = there && mine;
        const uint16_t* const b = lr.b + ((int64_t)id * N + n) * r;
        float low = 0.f;
        if constexpr (FUSED) {
            uint4 bv[kFusedRanks / 8];
#pragma unroll
            for (int k = 0; k < kFusedRanks; k += 8)
                if (adapt && k < r) bv[k / 8] = *reinterpret_cast<const uint4*>(b + k);
            lds_barrier();                                  // (s_h is there as well)
#pragma unroll
            for (int k = 0; k < kFusedRanks; k += 8) {
                if (!adapt || k >= r) continue;
                float hv[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) hv[i] = s_h[m * r + k + i];
                low = dot8f(hv, bv[k / 8], low);
            }
        } else {
            if (adapt) {
                const uint16_t* const h = lr.h + m * (2 * r);
#pragma unroll 4
                for (int k = 0; k < r; k += 8) {
                    const uint4 bv = *reinterpret_cast<const uint4*>(b + k);
                    low = dot8(*reinterpret_cast<const uint4*>(h + r + k), bv, low);
                    low = dot8(*reinterpret_cast<const uint4*>(h + k), bv, low);
                }
            }
            lds_barrier();
        }
        if (!there) continue;
        // row m, column at & 15 of the sixteen
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < FEW_WAVES; ++i)
            v += reinterpret_cast<const float*>(&s_sum[u & 1][i][(at & 15) / 4 * 16 + m])[at & 3];
        y[m * N + n] = (uint16_t)f32_to_bf16(v + low);
    }
}

}  // namespace

bool lora_fuses(int64_t M, int r) { return M * r <= kFusedRanks; }

hipError_t launch_lora_few(const uint16_t* x, int64_t M, int64_t K, const uint16_t* w, int64_t N, const LowRank& lr,
                           const uint16_t* a, const float* scale, uint16_t* y, hipStream_t s) {
    const bool fused = lora_fuses(M, lr.r);
    const dim3 block(few_threads(fused));
    // Wide layers, while a CU has three times sixteen columns (8192 columns, K = 4096, 16 rows:
    // 21.1 us without, 23.9) and enough of K for the two kinds of waves not to wait for each
    // other (12288 columns, K = 2048, r = 16: 4 rows 17.5 without, 20.1; 1 row 18.3 and 15.5)
    const int64_t cus = device_cu_count();
    if (K >= (fused ? 2048 : 4096) && N >= 48 * cus && M * wide_pitch(K) <= kWideX) {
        const dim3 wide((unsigned)cus);
        auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, wide, block, 0, s, x, M, K, w, N, lr, a, scale, y); };
        fused ? go(lora_wide_kernel<true>) : go(lora_wide_kernel<false>);
        return hipGetLastError();
    }
    // 16 columns a workgroup while that takes no more than two a CU (K = 4096, 16 rows, us:
    // N = 4096 15.4, with 32 columns 18.8; N = 8192 24.3 and 20.2; N = 14336 39.8 and 35.7)
    const int ct = N < 8192 ? 1 : 2;
    const dim3 grid((unsigned)((N + 16 * ct - 1) / (16 * ct)));
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, s, x, M, K, w, N, lr, a, scale, y); };
    if (fused) ct == 1 ? go(lora_few_kernel<1, true>) : go(lora_few_kernel<2, true>);
    else ct == 1 ? go(lora_few_kernel<1, false>) : go(lora_few_kernel<2, false>);
    return hipGetLastError();
}

// Where adapters have eight rows each on average, of 256 rows on two: the tiles add each
// adapter among 32 rows for itself.  4096 x 4096, 16 adapters of rank 64, us: 256 single rows
// 66 unsorted and 52 sorted, of rank 128 112 and 59; 64 adapters of rank 64, 400 rows 119 and
// 80; rank 16, 4096 rows 199 and 140.  Where each row's part is small (few_low_rank), only past
// 256 rows (rank 16, 400 rows of 64 adapters: 42 unsorted, 55).  Rows in 32-bit bytes; and up to
// 65536 of them, as one workgroup sorts (65600 single rows of 16 adapters, 4096 x 1024, unsorted:
// rank 16 1199, 65536 sorted 652; rank 128 7799 and 816).
bool lora_sorts(int64_t M, int64_t N, int64_t K, int L, int r) {
    const bool few = few_low_rank(M, N, r);
    return M > (few ? kLoraUnsorted : 64) && (few || M < 256 ? 8 : 2) * (int64_t)L <= M && M <= 65536 &&
           L <= kSortMaxL && M * K < ((int64_t)1 << 30);
}
hipError_t launch_lora_sort(const int32_t* ids, int64_t M, int L, int32_t* order, int32_t* sorted_ids,
                            int64_t* offs, hipStream_t s) {
    hipLaunchKernelGGL(lora_sort_kernel, dim3(1), dim3(SORT_THREADS), 0, s, ids, (int)M, L, order, sorted_ids, offs);
    return hipGetLastError();
}

hipError_t launch_lora_down(const LoraDown& p, hipStream_t s) {
    if (p.M == 0) return hipSuccess;
    if (p.order && p.M * p.r > kDownTiles) return launch_lora_down_tiles(p, s);
    const unsigned blocks = (unsigned)((p.M + 15) / 16), r = (unsigned)p.r;
    auto go = [&](auto kernel, dim3 grid) { hipLaunchKernelGGL(kernel, grid, dim3(64 * DOWN_WAVES), 0, s, p); };
    // one pass over x for up to 32 ranks, where 16 do not have too few workgroups
    const bool fine = !p.order && p.M * p.r <= kDownFine;
    if (r <= 16 || (!fine && blocks < 256))
        fine ? go(lora_down_kernel<1, true>, dim3(blocks, r / 4, 4)) : go(lora_down_kernel<1, false>, dim3(blocks, (r + 15) / 16, 2));
    else
        fine ? go(lora_down_kernel<2, true>, dim3(blocks, r / 4, 4))
             : go(lora_down_kernel<2, false>, dim3(blocks, (r + 31) / 32, 2));
    return hipGetLastError();
}

}  // namespace mx
