// bf16 products in 64 x 128 tiles (gfx950), for calls with few output tiles: the
// data and weight gradients of GroupedLinear and the adapter linear.
//
// One workgroup of four waves per tile and share of K; each wave owns 32 x 64 (two
// accumulators of the 32x32x16 MFMA).  K goes in steps of 64 through three LDS
// stages of 24 KB filled by direct loads two steps ahead, so two workgroups share a
// CU.  Where the tiles alone leave CUs idle, K is cut into `split` shares, whose
// fp32 sums go to memory and are added in order by a second launch: one order of
// every sum, no atomics.
//
// LDS orders (64 banks of 4 bytes): along K, chunk c of line n is stored at
// c ^ (n >> 1 & 7); across K, the 64-byte quarter of a row at quarter ^ (k & 3)
// (256-byte rows) or ^ (k >> 1 & 1) (128-byte rows), so that the rows that one
// transposing read takes lie on different banks.
#include "bf16_tiles.h"

namespace mx {
namespace {

constexpr int SM_M = 64, SM_N = 128, SM_K = 64, SM_ST = 3;
constexpr int SM_A = SM_M * 128, SM_B = SM_N * 128, SM_STAGE = SM_A + SM_B;
constexpr int SM_LOADS = 6;                        // per wave and step: 2 of A, 4 of B

struct SmallArgs {
    Bf16Problem p;
    int split;
};

// Rows [k0, k0 + 64) of an operand that lies across K: base at its first column,
// krows rows of ld values from there on, col0 columns to the left of the base.
__device__ __forceinline__ v4i across_rsrc(const uint16_t* p, int64_t k0, int64_t krows, int64_t ld,
                                           int64_t col0) {
    return make_rsrc(p + k0 * ld + col0, ((krows - k0) * ld - col0) * 2);
}

template <Bf16Form F>
__global__ void __launch_bounds__(256, 2)
bf16_small_kernel(SmallArgs s) {
    constexpr bool kA = F != Bf16Form::kWeightGrad;       // A lies along K
    constexpr bool kB = F == Bf16Form::kForward;          // B lies along K
    constexpr bool kRows = F != Bf16Form::kWeightGrad;    // groups own rows of C
    const Bf16Problem& p = s.p;
    __shared__ __attribute__((aligned(16))) uint8_t sm[SM_ST][SM_STAGE];
    __shared__ int s_prefix[kMaxGroups + 1];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int ntn = (int)((p.N + SM_N - 1) / SM_N);

    // ---- the workgroup's tile and share of K ----
    const int share = (int)(blockIdx.x % (unsigned)s.split);
    const int unit = (int)(blockIdx.x / (unsigned)s.split);
    int g;
    int64_t m0, mvalid, n0, row0 = 0, krows = p.K;
    if constexpr (F == Bf16Form::kForward) {
        g = 0;
        m0 = (int64_t)(unit / ntn) * SM_M;
        n0 = (int64_t)(unit % ntn) * SM_N;
        mvalid = p.M - m0;
    } else if constexpr (kRows) {
        // row tiles of each group: prefix sums (wave 0), then the unit's group
        if (wave == 0) {
            int cnt[kMaxGroups / 64], local = 0;
#pragma unroll
            for (int u = 0; u < kMaxGroups / 64; ++u) {
                const int i = lane * (kMaxGroups / 64) + u;
                int c = 0;
                if (i < p.G) {
                    const int64_t n = p.offs[i + 1] - p.offs[i];
                    c = n > 0 ? (int)((n + SM_M - 1) / SM_M) : 0;
                }
                cnt[u] = c;
                local += c;
            }
            int incl = local;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(incl, d);
                if (lane >= d) incl += o;
            }
            int run = incl - local;
#pragma unroll
            for (int u = 0; u < kMaxGroups / 64; ++u) {
                const int i = lane * (kMaxGroups / 64) + u;
                if (i < p.G) {
                    s_prefix[i] = run;
                    run += cnt[u];
                }
            }
            if (lane == 63) s_prefix[p.G] = incl;
        }
        __syncthreads();
        const int mt = unit / ntn;
        if (mt >= s_prefix[p.G]) return;
        int lo = 0, hi = p.G - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_prefix[mid] <= mt) lo = mid; else hi = mid - 1;
        }
        g = uni(lo);
        m0 = uni64(p.offs[g] + (int64_t)(mt - s_prefix[g]) * SM_M);
        n0 = (int64_t)(unit % ntn) * SM_N;
        mvalid = uni64(p.offs[g + 1]) - m0;
    } else {
        const int ntm = (int)((p.M + SM_M - 1) / SM_M);
        g = unit / (ntm * ntn);
        const int t = unit - g * (ntm * ntn);
        m0 = (int64_t)(t / ntn) * SM_M;
        n0 = (int64_t)(t % ntn) * SM_N;
        mvalid = p.M - m0;
        row0 = uni64(p.offs[g]);
        krows = uni64(p.offs[g + 1]) - row0;
        if (krows < 0) krows = 0;
    }
    mvalid = min(mvalid, (int64_t)SM_M);
    const int64_t nvalid = min(p.N - n0, (int64_t)SM_N);
    const int nk = (int)((krows + SM_K - 1) / SM_K);
    const int k_beg = (int)((int64_t)nk * share / s.split), k_end = (int)((int64_t)nk * (share + 1) / s.split);

    // ---- direct loads ----
    const int64_t lda = kA ? p.K : p.M, ldb = kB ? p.K : p.N;
    const uint16_t* const Bg = F == Bf16Form::kDataGrad ? p.B + (int64_t)g * p.K * p.N
                               : F == Bf16Form::kWeightGrad ? p.B + row0 * p.N : p.B;
    const uint16_t* const Ag = F == Bf16Form::kWeightGrad ? p.A + row0 * p.M : p.A;
    const v4i ra = make_rsrc(Ag + m0 * lda, mvalid * lda * 2);     // (along K)
    const v4i rb = make_rsrc(Bg + n0 * ldb, nvalid * ldb * 2);
    const uint32_t smb = (uint32_t)uni((int)lds_addr(sm));
    auto load = [&](int ks) {
        const bool live = ks < k_end;
        const uint32_t at = smb + (uint32_t)((ks - k_beg) % SM_ST) * SM_STAGE;
        auto rng = [&](const v4i& r) { return live ? r : v4i{r.x, r.y, 0, r.w}; };
        const int64_t left = p.K - (int64_t)ks * SM_K;     // K values of the step (along K)
        if constexpr (kA) {
            static_for<2>([&](auto uc) {
                constexpr int u = decltype(uc)::value;
                const int row = wave * 16 + u * 8 + (lane >> 3);
                const int c = (lane & 7) ^ ((row >> 1) & 7);
                const uint32_t off = (uint32_t)(row * lda * 2) + (uint32_t)c * 16u;
                dma_b128<u * 1024>(rng(ra), at + wave * 2048, off | (c * 8 < left ? 0u : 0x80000000u),
                                   (uint32_t)ks * 128u);
            });
        } else {
            const v4i r = rng(across_rsrc(Ag, (int64_t)ks * SM_K, krows, lda, m0));
            static_for<2>([&](auto uc) {
                constexpr int u = decltype(uc)::value;
                const int k = wave * 16 + u * 8 + (lane >> 3);
                const int c = (lane & 7) ^ (((k >> 1) & 1) << 2);
                dma_b128<u * 1024>(r, at + wave * 2048, (uint32_t)(k * lda * 2) + (uint32_t)c * 16u, 0u);
            });
        }
        if constexpr (kB) {
            static_for<4>([&](auto uc) {
                constexpr int u = decltype(uc)::value;
                const int row = wave * 32 + u * 8 + (lane >> 3);
                const int c = (lane & 7) ^ ((row >> 1) & 7);
                const uint32_t off = (uint32_t)(row * ldb * 2) + (uint32_t)c * 16u;
                dma_b128<u * 1024>(rng(rb), at + SM_A + wave * 4096, off | (c * 8 < left ? 0u : 0x80000000u),
                                   (uint32_t)ks * 128u);
            });
        } else {
            const v4i r = rng(across_rsrc(Bg, (int64_t)ks * SM_K, krows, ldb, n0));
            static_for<4>([&](auto uc) {
                constexpr int u = decltype(uc)::value;
                const int k = wave * 16 + u * 4 + (lane >> 4);
                const int c = (lane & 15) ^ ((k & 3) << 2);
                dma_b128<u * 1024>(r, at + SM_A + wave * 4096, (uint32_t)(k * ldb * 2) + (uint32_t)c * 16u, 0u);
            });
        }
    };

    // ---- fragments ----
    const int l32 = lane & 31, half = lane >> 5;
    auto frag_a = [&](const uint8_t* st, int kk) -> bf16x8 {
        if constexpr (kA) {
            const int row = wm * 32 + l32;
            return frag_along(st + row * 128 + (((2 * kk + half) ^ ((row >> 1) & 7)) << 4));
        } else {
            const int k = 16 * kk + 8 * half + ((lane >> 2) & 3);
            const int c = (wm * 4 + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ (((k >> 1) & 1) << 2);
            return frag_across(st + k * 128 + (c << 4) + 8 * (lane & 1), 4 * 128);
        }
    };
    auto frag_b = [&](const uint8_t* st, int j, int kk) -> bf16x8 {
        if constexpr (kB) {
            const int row = wn * 64 + j * 32 + l32;
            return frag_along(st + SM_A + row * 128 + (((2 * kk + half) ^ ((row >> 1) & 7)) << 4));
        } else {
            const int k = 16 * kk + 8 * half + ((lane >> 2) & 3);
            const int c = (wn * 8 + j * 4 + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ ((k & 3) << 2);
            return frag_across(st + SM_A + k * 256 + (c << 4) + 8 * (lane & 1), 4 * 256);
        }
    };

    v16f acc[2] = {zero16(), zero16()};
    for (int ks = k_beg; ks < k_beg + SM_ST - 1; ++ks) load(ks);
    for (int ks = k_beg; ks < k_end; ++ks) {
        wait_vm<(SM_ST - 2) * SM_LOADS>();     // this wave's loads of step ks have landed
        lds_barrier();                         // and everybody's; step ks - 1 is read
        load(ks + SM_ST - 1);
        const uint8_t* const st = sm[(ks - k_beg) % SM_ST];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const bf16x8 a = frag_a(st, kk);
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[j] = mfma_bf16(frag_b(st, j, kk), a, acc[j]);
        }
    }
    wait_vm<0>();          // no load may still be landing in LDS when the workgroup ends

    // ---- output: the wave's 32 x 64 ----
    const int64_t rw = m0 + wm * 32, cw = n0 + wn * 64;
    const int rows = (int)(mvalid - wm * 32), cols = (int)(nvalid - wn * 64);
    if (F == Bf16Form::kForward && p.lr.r && share == s.split - 1) {
        const bool there = l32 < rows;
        int id = there ? p.lr.id[rw + l32] : -1;
        if (id >= p.lr.L) id = -1;
        add_adapters<2>(acc, p.lr, there ? p.lr.h + (rw + l32) * (2 * p.lr.r) : nullptr, id, p.N, cw, lane);
    }
    const int64_t gstride = kRows ? 0 : p.M * p.N;       // C of each group
    if (s.split > 1) {
        const int64_t all = (kRows ? p.rows : (int64_t)p.G * p.M) * p.N;
        float* const part = p.parts + share * all + g * gstride;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            store_f32_32x32<false>(acc[j], reinterpret_cast<uint8_t*>(part + rw * p.N + cw + 32 * j), p.N * 4,
                                   rows, cols - 32 * j, lane);
        return;
    }
    if constexpr (F == Bf16Form::kWeightGrad) {
        if (p.c_f32) {
            float* const c = static_cast<float*>(p.C) + g * gstride + rw * p.N + cw;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint8_t* const at = reinterpret_cast<uint8_t*>(c + 32 * j);
                if (p.c_add) store_f32_32x32<true>(acc[j], at, p.N * 4, rows, cols - 32 * j, lane);
                else store_f32_32x32<false>(acc[j], at, p.N * 4, rows, cols - 32 * j, lane);
            }
            return;
        }
    }
    uint8_t* const at = reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.C) + g * gstride + rw * p.N + cw);
    if (F == Bf16Form::kDataGrad && p.rscale) {
        const bool there = l32 < rows;
        if (p.drp && cols > 0) {
            const uint16_t* const xr = there ? p.drx + (rw + l32) * p.N + cw : nullptr;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) sum += dot_32(acc[j], xr ? xr + 32 * j : nullptr, cols - 32 * j, lane);
            sum += __shfl_xor(sum, 32);
            if (there && half == 0) p.drp[(cw / 64) * p.M + rw + l32] = sum;
        }
        store_bf16_32x64<true>(acc[0], acc[1], there ? p.rscale[rw + l32] : 0.f, at, (uint32_t)p.N * 2u, rows,
                               cols, lane);
        return;
    }
    store_bf16_32x64<false>(acc[0], acc[1], 1.f, at, (uint32_t)p.N * 2u, rows, cols, lane);
}

// ---- sums of the shares ------------------------------------------------------------
__device__ __forceinline__ void sum_parts8(const float* parts, int64_t all, int split, int64_t i, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
    for (int c = 0; c < split; ++c) {
        const float4* q = reinterpret_cast<const float4*>(parts + c * all + i);
        const float4 a = q[0], b = q[1];
        v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
}

// Eight values a thread.
__global__ void __launch_bounds__(256)
bf16_join_kernel(const float* __restrict__ parts, int64_t all, int split, void* __restrict__ c, bool f32,
                 bool add) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= all) return;
    float v[8];
    sum_parts8(parts, all, split, i, v);
    if (!f32) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(c) + i) = pack8(v);
        return;
    }
    float* const out = static_cast<float*>(c) + i;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
        float4 y = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        if (add) {
            const float4 o = *reinterpret_cast<const float4*>(out + e);
            y = make_float4(o.x + y.x, o.y + y.y, o.z + y.z, o.w + y.w);
        }
        *reinterpret_cast<float4*>(out + e) = y;
    }
}

// One row a workgroup, with its factor and (dr given) dr[row] = x . (the row without it).
__global__ void __launch_bounds__(256)
bf16_join_rows_kernel(const float* __restrict__ parts, int64_t M, int64_t N, int split,
                      const float* __restrict__ rscale, const uint16_t* __restrict__ x,
                      uint16_t* __restrict__ c, float* __restrict__ dr) {
    const int64_t row = blockIdx.x;
    const float sc = rscale[row];
    float sum = 0.f;
    for (int64_t n = threadIdx.x * 8; n < N; n += 2048) {
        float v[8];
        sum_parts8(parts, M * N, split, row * N + n, v);
        uint4 xv = make_uint4(0, 0, 0, 0);
        if (dr) xv = *reinterpret_cast<const uint4*>(x + row * N + n);
        const uint32_t w[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sum += v[2 * e] * bf16_to_f32(w[e] & 0xffffu) + v[2 * e + 1] * __uint_as_float(w[e] & 0xffff0000u);
            v[2 * e] *= sc;
            v[2 * e + 1] *= sc;
        }
        *reinterpret_cast<uint4*>(c + row * N + n) = pack8(v);
    }
    if (!dr) return;
    __shared__ float s_sum[4];
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) dr[row] = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
}

__global__ void __launch_bounds__(256)
scale_rows_kernel(const uint16_t* __restrict__ x, const float* __restrict__ r, int64_t M, int C8,
                  uint16_t* __restrict__ out) {
    // rows by grid, a row's 16-byte pieces by thread
    for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
        const float sc = r[row];
        for (int c = threadIdx.x; c < C8; c += 256) {
            const int64_t i = row * C8 + c;
            const uint4 v = *reinterpret_cast<const uint4*>(x + i * 8);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            float f[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[2 * e] = bf16_to_f32(w[e] & 0xffffu) * sc;
                f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u) * sc;
            }
            *reinterpret_cast<uint4*>(out + i * 8) = pack8(f);
        }
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of a call (an upper bound where groups own rows: their counts are on the device).
int64_t small_tiles(const Bf16Problem& p) {
    const int64_t ntn = cdiv(p.N, SM_N);
    if (p.form == Bf16Form::kForward) return cdiv(p.M, SM_M) * ntn;
    if (p.form == Bf16Form::kDataGrad)       // sum of ceil(rows / 64) <= this
        return (p.rows < p.G ? p.rows : p.G + (p.rows - p.G) / SM_M) * ntn;
    return (int64_t)p.G * cdiv(p.M, SM_M) * ntn;
}

int small_split(const Bf16Problem& p) {
    const int64_t tiles = small_tiles(p);
    // a group's steps of K, by the average
    const int64_t nk = cdiv(p.form == Bf16Form::kWeightGrad ? cdiv(p.rows, p.G) : p.K, SM_K);
    int64_t split = tiles ? 512 / tiles : 1;
    if (split > nk / 4) split = nk / 4;
    return split < 1 ? 1 : split > 16 ? 16 : (int)split;
}

}  // namespace

int64_t bf16_parts(const Bf16Problem& p) {
    const int split = small_split(p);
    return split > 1 ? split * (p.form == Bf16Form::kWeightGrad ? (int64_t)p.G * p.M : p.rows) * p.N : 0;
}

int64_t bf16_product_tiles(const Bf16Problem& p) { return small_tiles(p) * small_split(p); }

int64_t bf16_dr_parts(int64_t N) { return cdiv(N, 64); }

hipError_t launch_bf16_product(const Bf16Problem& p, hipStream_t st) {
    SmallArgs a{p, small_split(p)};
    const int64_t grid = small_tiles(p) * a.split;
    if (grid == 0) return hipSuccess;
    const dim3 gd((unsigned)grid), bd(256);
    switch (p.form) {
        case Bf16Form::kForward: hipLaunchKernelGGL(bf16_small_kernel<Bf16Form::kForward>, gd, bd, 0, st, a); break;
        case Bf16Form::kDataGrad: hipLaunchKernelGGL(bf16_small_kernel<Bf16Form::kDataGrad>, gd, bd, 0, st, a); break;
        default: hipLaunchKernelGGL(bf16_small_kernel<Bf16Form::kWeightGrad>, gd, bd, 0, st, a);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.split > 1) {
        if (p.rscale) {
            hipLaunchKernelGGL(bf16_join_rows_kernel, dim3((unsigned)p.M), bd, 0, st, p.parts, p.M, p.N, a.split,
                               p.rscale, p.drx, static_cast<uint16_t*>(p.C), p.dr);
        } else {
            const int64_t all = (p.form == Bf16Form::kWeightGrad ? (int64_t)p.G * p.M : p.rows) * p.N;
            hipLaunchKernelGGL(bf16_join_kernel, dim3((unsigned)cdiv(all, 2048)), bd, 0, st, p.parts, all, a.split,
                               p.C, p.c_f32, p.c_add);
        }
        return hipGetLastError();
    }
    if (p.drp) return launch_dr_reduce(p.drp, p.M, bf16_dr_parts(p.N), p.dr, st);
    return hipSuccess;
}

hipError_t launch_scale_rows(const uint16_t* x, const float* r, int64_t M, int64_t C, uint16_t* out,
                             hipStream_t s) {
    if (M == 0) return hipSuccess;
    hipLaunchKernelGGL(scale_rows_kernel, dim3((unsigned)(M < 65536 ? M : 65536)), dim3(256), 0, s, x, r, M,
                       (int)(C / 8), out);
    return hipGetLastError();
}

}  // namespace mx
