// bf16 products in small (64 x 128) and middle (128 x 128) tiles (gfx950), for calls with
// few output tiles and what rounds of large ones leave, and the choice between them: the
// data and weight gradients of GroupedLinear and the adapter linear.
//
// One workgroup of four waves per tile and share of K; each wave owns 32 RB x 64 (RB x 2
// accumulators of the 32x32x16 MFMA).  K goes in steps of 64 through LDS stages filled by
// direct loads.  A step's fragments are read into registers all along the step before it,
// so one barrier a step is enough: behind it the next step's stage has landed and this
// step's, already read, is refilled.  (With the reads in the half of a step that follows
// a second barrier, as registers allow the large kernel, that half is bound by the LDS:
// 6 to 10 % slower here.)  Two workgroups share a CU and hide each other's waits, with three
// stages (small tiles) or two (middle ones); a launch of at most one middle tile a CU takes
// four (1024 rows of 4096 x 4096: 38 us, with two stages 47).  Loading a middle tile's step
// takes a CU 0.25 us, its MFMAs 0.21 and the LDS about as long, and one wave a SIMD has to
// issue all of it: 0.48 us.  So the code of a step holds nothing that could be left out:
// stages are constants (75 instructions for 16 MFMAs; with stages counted, 127 and 0.56
// us), and the end of K is dealt with once, in the last step.  Where the tiles alone leave
// CUs idle, K is cut into `split` shares, whose fp32 sums go to memory and are added in
// order by a second launch: one order of every sum, no atomics.
//
// LDS orders (64 banks of 4 bytes): along K, chunk c of line n is stored at
// c ^ (n >> 1 & 7); across K, the 64-byte quarter of a 256-byte row at quarter ^ (k & 3),
// so that the rows that one transposing read takes lie on different banks.
#include "lora_down.h"

namespace mx {
namespace {

// MB: 32-row blocks of a wave (1: tiles of 64 x 128, 2: of 128 x 128).
constexpr int SM_N = 128, SM_K = 64, SM_B = SM_N * 128;
constexpr int small_m(int MB) { return 64 * MB; }

struct SmallArgs {
    Bf16Problem p;
    int split;
    bool lr_here;          // the tiles add the adapters' part (else the join)
    int rounds;            // > 0: only the tiles that the large kernel with that many workgroups left
};

// Rows [k0, k0 + 64) of an operand that lies across K: base at its first column,
// krows rows of ld values from there on, col0 columns to the left of the base.
__device__ __forceinline__ v4i across_rsrc(const uint16_t* p, int64_t k0, int64_t krows, int64_t ld,
                                           int64_t col0) {
    return make_rsrc(p + k0 * ld + col0, ((krows - k0) * ld - col0) * 2);
}

constexpr int small_stage(int MB) { return small_m(MB) * 128 + SM_B; }
constexpr int per_cu(int MB, int ST) { return 2 * ST * small_stage(MB) <= 160 * 1024 ? 2 : 1; }

// What workgroup `block` (of a multiple of 128) of a product's does.
template <Bf16Form F, int MB, int ST>
__device__ __forceinline__ void small_tile(const SmallArgs& s, const int block,
                                           uint8_t (&sm)[ST][small_stage(MB)]) {
    constexpr int SM_M = small_m(MB), SM_A = SM_M * 128, SM_STAGE = small_stage(MB);
    constexpr int SM_LOADS = 2 * MB + 4;                  // per wave and step, of A and B
    constexpr int SLOTS = 8 * MB, READS = 4 * (MB + 2);   // of a step: MFMAs, fragments
    constexpr int WAIT = MB;                          // MFMAs before its barrier
    constexpr bool kA = F != Bf16Form::kWeightGrad;       // A lies along K
    constexpr bool kB = F == Bf16Form::kForward || F == Bf16Form::kDown;         // B lies along K
    constexpr bool kRows = F != Bf16Form::kWeightGrad;    // groups own rows of C
    constexpr bool kGroups = F == Bf16Form::kDataGrad || F == Bf16Form::kDown;   // more than one
    const Bf16Problem& p = s.p;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int ntn = (int)((p.N + SM_N - 1) / SM_N);

    // ---- the workgroup's tile and share of K ----
    int g = 0;
    int64_t m0, mvalid, n0, row0 = 0, krows = p.K;
    // tiles there are (the grid may be larger: the rows of groups are on the device)
    const bool rest = kRows && MB == 2 && s.rounds;       // quarters of what the large kernel left
    const int ntl = (int)((p.N + 255) / 256);
    int mtiles = 0, units, left = 0;
    if constexpr (kGroups)
        mtiles = rest ? count_row_tiles<256>(p.offs, p.G, lane) : count_row_tiles<SM_M>(p.offs, p.G, lane);
    else
        mtiles = (int)((p.M + (rest ? 256 : SM_M) - 1) / (rest ? 256 : SM_M));
    if (rest) {
        left = whole_rounds(mtiles * ntl, s.rounds);
        units = (mtiles * ntl - left) * 4;
    } else {
        units = mtiles * ntn * (kRows ? 1 : p.G) * s.split;
    }
    // workgroup b runs on XCD b % 8: each XCD takes 16 tiles of a band at a time, so that
    // those it runs together share panels in its L2 and long sums are spread over all XCDs
    const int nth = block / 8, at = nth / 16 * 128 + block % 8 * 16 + nth % 16;
    if (at >= units) return;
    const int share = at % s.split, unit = at / s.split;
    if constexpr (kRows) {
        RowGroup rg{0, 0, mtiles, 0, p.M};
        int mt, nt;
        if (rest) {
            const int t = left + unit / 4;
            if constexpr (kGroups) rg = find_row_group<256>(p.offs, p.G, t / ntl, lane);
            const TileAt to = band_order(t - rg.first * ntl, rg.tiles, ntl);
            mt = to.m * 2 + (unit >> 1 & 1);
            nt = to.n * 2 + (unit & 1);
            if (nt >= ntn) return;
        } else {
            if constexpr (kGroups) rg = find_row_group<SM_M>(p.offs, p.G, unit / ntn, lane);
            const TileAt to = band_order(unit - rg.first * ntn, rg.tiles, ntn);
            mt = to.m;
            nt = to.n;
        }
        g = rg.g;
        m0 = rg.row0 + (int64_t)mt * SM_M;
        n0 = (int64_t)nt * SM_N;
        mvalid = rg.rows - (int64_t)mt * SM_M;
        if (mvalid <= 0) return;
    } else {
        g = unit / (mtiles * ntn);
        const TileAt to = band_order(unit - g * (mtiles * ntn), mtiles, ntn);
        m0 = (int64_t)to.m * SM_M;
        n0 = (int64_t)to.n * SM_N;
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
    const uint16_t* const Bg = kGroups ? p.B + (int64_t)g * p.K * p.N
                               : F == Bf16Form::kWeightGrad ? p.B + row0 * p.N : p.B;
    const uint16_t* const Ag = F == Bf16Form::kWeightGrad ? p.A + row0 * p.M : p.A;
    // (along K; the adapter linear may take its rows in another order)
    const int32_t* const order = F == Bf16Form::kForward || F == Bf16Form::kDown ? p.lr.order : nullptr;
    const v4i ra = order ? make_rsrc(Ag, p.M * lda * 2) : make_rsrc(Ag + m0 * lda, mvalid * lda * 2);
    const v4i rb = make_rsrc(Bg + n0 * ldb, nvalid * ldb * 2);
    const uint32_t smb = (uint32_t)uni((int)lds_addr(sm));
    // a lane's offsets: along K 8 rows a load (odd loads' chunks are the even ones' ^ 4),
    // across K rows of 256 bytes
    uint32_t aoff[2 * MB], boff, bflip = 0;
    const int ac = (lane & 7) ^ (lane >> 4);              // chunk of an even load along K
    if constexpr (kA) {
#pragma unroll
        for (int u = 0; u < 2 * MB; ++u) {
            const int row = wave * (16 * MB) + u * 8 + (lane >> 3);
            const int64_t from = !order ? row : row < mvalid ? order[m0 + row] : -1;
            aoff[u] = (from < 0 ? 0x80000000u : (uint32_t)(from * lda * 2)) + (uint32_t)(ac ^ (u & 1 ? 4 : 0)) * 16u;
        }
    } else {
        static_assert(kA || MB == 2, "256-byte rows of A across K");
#pragma unroll
        for (int u = 0; u < 2 * MB; ++u) {
            const int k = wave * 16 + u * 4 + (lane >> 4), c = (lane & 15) ^ ((k & 3) << 2);
            aoff[u] = (uint32_t)(k * lda * 2) + (uint32_t)c * 16u;
        }
    }
    if constexpr (kB) {
        boff = (uint32_t)((wave * 32 + (lane >> 3)) * ldb * 2) + (uint32_t)ac * 16u;
        bflip = (ac & 4) ? (uint32_t)-64 : 64u;
    } else {
        const int k = wave * 16 + (lane >> 4), c = (lane & 15) ^ ((k & 3) << 2);
        boff = (uint32_t)(k * ldb * 2) + (uint32_t)c * 16u;
    }
    const uint32_t brow = (uint32_t)((kB ? 8 : 4) * ldb * 2);
    struct Rsrc {
        v4i a, b;
        uint32_t soff;
    };
    // descriptors of step ks.  (Along K the lanes of a last step whose chunk lies past K
    // load what follows; its MFMAs leave that out.)
    auto rsrc_of = [&](int ks) -> Rsrc {
        Rsrc r{kA ? ra : across_rsrc(Ag, (int64_t)ks * SM_K, krows, lda, m0),
               kB ? rb : across_rsrc(Bg, (int64_t)ks * SM_K, krows, ldb, n0), (uint32_t)ks * 128u};
        r.a.z = ks < k_end ? r.a.z : 0;
        r.b.z = ks < k_end ? r.b.z : 0;
        return r;
    };
    auto dma = [&](auto uc, const Rsrc& r, int st) {
        constexpr int u = decltype(uc)::value;
        const uint32_t at = smb + (uint32_t)st * SM_STAGE;
        if constexpr (u < 2 * MB) {
            dma_b128<u * 1024>(r.a, at + wave * (2048 * MB), aoff[u], kA ? r.soff : 0u);
        } else {
            constexpr int v = u - 2 * MB;
            dma_b128<v * 1024>(r.b, at + SM_A + wave * 4096, boff + v * brow + (v & 1 ? bflip : 0u), kB ? r.soff : 0u);
        }
    };

    // ---- fragments ----
    const int l32 = lane & 31, half = lane >> 5;
    auto frag_a = [&](const uint8_t* st, int i, int kk) -> bf16x8 {
        if constexpr (kA) {
            const int row = wm * (32 * MB) + i * 32 + l32;
            return frag_along(st + row * 128 + (((2 * kk + half) ^ ((row >> 1) & 7)) << 4));
        } else {
            const int k = 16 * kk + 8 * half + ((lane >> 2) & 3);
            const int c = ((wm * 2 + i) * 4 + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ ((k & 3) << 2);
            return frag_across(st + k * 256 + (c << 4) + 8 * (lane & 1), 4 * 256);
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

    v16f acc[MB][2];
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[i][0] = acc[i][1] = zero16();
    // A step's fragments are read during the one before it, all along it, so its stage is
    // free when it begins.
    struct Frags {
        bf16x8 a[MB][4], b[2][4];
    };
    auto read = [&](auto nc, Frags& f, const uint8_t* st) {      // in the order of their use
        constexpr int n = decltype(nc)::value, kk = n / (MB + 2), w = n % (MB + 2);
        if constexpr (w < 2) f.b[w][kk] = frag_b(st, w, kk);
        else f.a[w - 2][kk] = frag_a(st, w - 2, kk);
    };
    auto step = [&](auto stc, int ks, Frags& cur, Frags& nxt) {
        constexpr int st = decltype(stc)::value;
        const Rsrc r = rsrc_of(ks + ST);
        static_for<SLOTS>([&](auto tc) {
            constexpr int t = decltype(tc)::value, kk = t / (2 * MB), i = t / 2 % MB, j = t % 2;
            constexpr int at = t - WAIT;          // of the slots behind the barrier
            if constexpr (at == 0) {
                wait_vm<(ST - 2) * SM_LOADS>();   // this wave's loads of step ks + 1 have landed
                lds_barrier();                    // and everybody's, and this step's stage is read
            }
            acc[i][j] = mfma_bf16(cur.b[j][kk], cur.a[i][kk], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (at >= 0) {
                // spread evenly (no read in the last slot)
                constexpr int RS = SLOTS - WAIT - 1, LS = SLOTS - WAIT;
                static_for<(READS + RS - 1) / RS>([&](auto uc) {
                    constexpr int n = (at * READS + RS - 1) / RS + decltype(uc)::value;
                    if constexpr (n < READS && n * RS < (at + 1) * READS)
                        read(std::integral_constant<int, n>{}, nxt, sm[(st + 1) % ST]);
                });
                static_for<(SM_LOADS + LS - 1) / LS>([&](auto uc) {
                    constexpr int n = (at * SM_LOADS + LS - 1) / LS + decltype(uc)::value;
                    if constexpr (n < SM_LOADS && n * LS < (at + 1) * SM_LOADS)
                        dma(std::integral_constant<int, n>{}, r, st);
                });
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // The last one: sixteens of K up to the end of an operand along K (others are zeros).
    auto last = [&](const Frags& cur) {
        const int64_t left = p.K - (int64_t)(k_end - 1) * SM_K;
        static_for<4>([&](auto kc) {
            constexpr int kk = decltype(kc)::value;
            if (kk > 0 && kA && 16 * kk >= left) return;
            static_for<MB>([&](auto ic) {
                constexpr int i = decltype(ic)::value;
                acc[i][0] = mfma_bf16(cur.b[0][kk], cur.a[i][kk], acc[i][0]);
                acc[i][1] = mfma_bf16(cur.b[1][kk], cur.a[i][kk], acc[i][1]);
            });
        });
    };
    // Steps go in pairs, with stages that the code holds as constants, up to one that is
    // left: with an even number of them the first goes alone, in the last stage.
    Frags f0, f1;
    const bool even = ((k_end - k_beg) & 1) == 0;
    auto fill = [&](int i) {                      // step k_beg + i
        const Rsrc r = rsrc_of(k_beg + i);
        const int st = even ? (i + ST - 1) % ST : i;
        static_for<SM_LOADS>([&](auto uc) { dma(uc, r, st); });
    };
    fill(0);
    if (k_beg + 1 < k_end) {
#pragma unroll
        for (int i = 1; i < ST; ++i) fill(i);
        wait_vm<(ST - 1) * SM_LOADS>();
    } else {
        wait_vm<0>();
    }
    lds_barrier();
    int ks = k_beg;
    if (even) {
        static_for<READS>([&](auto nc) { read(nc, f1, sm[ST - 1]); });
        if (ks < k_end) step(std::integral_constant<int, ST - 1>{}, ks++, f1, f0);
    } else {
        static_for<READS>([&](auto nc) { read(nc, f0, sm[0]); });
    }
    while (ks + 1 < k_end) {
        static_for<ST % 2 ? ST : ST / 2>([&](auto uc) {
            constexpr int u = 2 * decltype(uc)::value;
            if (u && ks + 1 >= k_end) return;
            step(std::integral_constant<int, u % ST>{}, ks, f0, f1);
            step(std::integral_constant<int, (u + 1) % ST>{}, ks + 1, f1, f0);
            ks += 2;
        });
    }
    if (ks < k_end) last(f0);
    wait_vm<0>();          // no load may still be landing in LDS when the workgroup ends

    // ---- output: the wave's blocks of 32 x 64 ----
    const int64_t gstride = kRows ? 0 : p.M * p.N;       // C of each group
    const int64_t cw = n0 + wn * 64;
    const int cols = (int)(nvalid - wn * 64);
    static_for<MB>([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        const int64_t rw = m0 + (wm * MB + i) * 32;
        const int rows = (int)(mvalid - (wm * MB + i) * 32);
        const bool there = l32 < rows;
        v16f (&av)[2] = acc[i];
        if (F == Bf16Form::kForward && s.lr_here && share == s.split - 1) {
            int id = there ? p.lr.id[rw + l32] : -1;
            if (id >= p.lr.L) id = -1;
            add_adapters<2, 4>(av, p.lr, there ? p.lr.h + (rw + l32) * (2 * p.lr.r) : nullptr, id, p.N, cw, lane);
        }
        if (s.split > 1) {
            const int64_t all = (kRows ? p.rows : (int64_t)p.G * p.M) * p.N;
            float* const part = p.parts + share * all + g * gstride;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                store_f32_32x32<false>(av[j], reinterpret_cast<uint8_t*>(part + rw * p.N + cw + 32 * j), p.N * 4,
                                       rows, cols - 32 * j, lane);
            return;
        }
        if (F == Bf16Form::kWeightGrad && p.c_f32) {
            float* const c = static_cast<float*>(p.C) + g * gstride + rw * p.N + cw;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint8_t* const at = reinterpret_cast<uint8_t*>(c + 32 * j);
                if (p.c_add) store_f32_32x32<true>(av[j], at, p.N * 4, rows, cols - 32 * j, lane);
                else store_f32_32x32<false>(av[j], at, p.N * 4, rows, cols - 32 * j, lane);
            }
            return;
        }
        if constexpr (F == Bf16Form::kDown) {
            const float sc = p.rscale ? p.rscale[g] : 1.f;
            v16f lo[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    uint32_t h, l;
                    split2(av[j][v] * sc, h, l);
                    av[j][v] = bf16_to_f32(h);
                    lo[j][v] = bf16_to_f32(l);
                }
            uint8_t* const to = reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.C) + rw * (2 * p.N) + cw);
            store_bf16_32x64<false>(av[0], av[1], 1.f, to, (uint32_t)p.N * 4u, rows, cols, lane);
            store_bf16_32x64<false>(lo[0], lo[1], 1.f, to + p.N * 2, (uint32_t)p.N * 4u, rows, cols, lane);
            return;
        }
        uint8_t* const at = reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.C) + g * gstride + rw * p.N + cw);
        if (F == Bf16Form::kDataGrad && p.rscale) {
            if (p.drp && cols > 0) {
                const uint16_t* const xr = there ? p.drx + (rw + l32) * p.N + cw : nullptr;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 2; ++j) sum += dot_32(av[j], xr ? xr + 32 * j : nullptr, cols - 32 * j, lane);
                sum += __shfl_xor(sum, 32);
                if (there && half == 0) p.drp[(cw / 64) * p.M + rw + l32] = sum;
            }
            store_bf16_32x64<true>(av[0], av[1], there ? p.rscale[rw + l32] : 0.f, at, (uint32_t)p.N * 2u, rows, cols,
                                   lane);
            return;
        }
        if constexpr (F == Bf16Form::kForward) {
            int to[4];
            line_rows(to, order, rw, rows, lane);
            store_bf16_32x64<false, true>(av[0], av[1], 1.f, reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.C) + cw),
                                          (uint32_t)p.N * 2u, rows, cols, lane, to);
        } else {
            store_bf16_32x64<false>(av[0], av[1], 1.f, at, (uint32_t)p.N * 2u, rows, cols, lane);
        }
    });
}

template <int MB, int ST>
__global__ void __launch_bounds__(256, per_cu(MB, ST))
bf16_forward_kernel(SmallArgs s) {
    __shared__ __attribute__((aligned(16))) uint8_t sm[ST][small_stage(MB)];
    small_tile<Bf16Form::kForward, MB, ST>(s, (int)blockIdx.x, sm);
}

// The same with the adapters' down projection in the workgroups from `tiles` on, for calls
// whose join adds the adapters' part.
template <int MB, int ST>
__global__ void __launch_bounds__(256, per_cu(MB, ST))
bf16_forward_down_kernel(SmallArgs s, LoraDown d, int tiles) {
    union Smem {
        uint8_t tile[ST][small_stage(MB)];
        v4f sum[4][1][64];
    };
    __shared__ __attribute__((aligned(16))) Smem sm;
    const int b = (int)blockIdx.x - tiles, ranks = d.r / 4;
    if (b < 0) return small_tile<Bf16Form::kForward, MB, ST>(s, (int)blockIdx.x, sm.tile);
    lora_down<4, 1, true>(d, b / (4 * ranks), b / 4 % ranks, b % 4, sm.sum);
}

// The adapters' down projection of sorted rows, adapters as groups.
__global__ void __launch_bounds__(256, 2)
bf16_down_kernel(SmallArgs s) {
    __shared__ __attribute__((aligned(16))) uint8_t sm[3][small_stage(1)];
    small_tile<Bf16Form::kDown, 1, 3>(s, (int)blockIdx.x, sm);
}

// ---- sums of the shares ------------------------------------------------------------
template <int V>           // consecutive values: 4 or 8
__device__ __forceinline__ void sum_parts(const float* parts, int64_t all, int split, int64_t i, float (&v)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = 0.f;
#pragma unroll 8
    for (int c = 0; c < split; ++c) {
        const float4* q = reinterpret_cast<const float4*>(parts + c * all + i);
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            const float4 a = q[e / 4];
            v[e] += a.x; v[e + 1] += a.y; v[e + 2] += a.z; v[e + 3] += a.w;
        }
    }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
}

// Four values a thread.
__global__ void __launch_bounds__(256)
bf16_join_kernel(const float* __restrict__ parts, int64_t all, int split, void* __restrict__ c, bool f32,
                 bool add) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= all) return;
    float v[4];
    sum_parts(parts, all, split, i, v);
    if (!f32) {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c) + i) = pack4_bf16(v);
        return;
    }
    float4* const out = reinterpret_cast<float4*>(static_cast<float*>(c) + i);
    float4 y = make_float4(v[0], v[1], v[2], v[3]);
    if (add) {
        const float4 o = *out;
        y = make_float4(o.x + y.x, o.y + y.y, o.z + y.z, o.w + y.w);
    }
    *out = y;
}

// Four columns of a row a thread (rows by grid.y), for the adapter linear: rows to where
// they belong, and (ADAPTERS) the adapters' part, each value the dot of the row's h with
// its adapter's row of b.
template <bool ADAPTERS>
__global__ void __launch_bounds__(256)
bf16_join_adapters_kernel(const float* __restrict__ parts, int64_t M, int64_t N, int split, LowRank lr,
                          uint16_t* __restrict__ c) {
    const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (n >= N) return;
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
        float low[4] = {0.f, 0.f, 0.f, 0.f};
        if constexpr (ADAPTERS) {
            const int id = lr.id[m], r = lr.r;
            if (id >= 0 && id < lr.L) {
                const uint16_t* const h = lr.h + m * (2 * r);
                const uint16_t* const b = lr.b + ((int64_t)id * N + n) * r;
#pragma unroll 2
                for (int k = 0; k < r; k += 8) {
                    const uint4 hi = *reinterpret_cast<const uint4*>(h + k), lo = *reinterpret_cast<const uint4*>(h + r + k);
                    const uint32_t hw[4] = {hi.x, hi.y, hi.z, hi.w}, lw[4] = {lo.x, lo.y, lo.z, lo.w};
                    uint4 bv[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) bv[e] = *reinterpret_cast<const uint4*>(b + e * r + k);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float h0 = bf16_to_f32(hw[q] & 0xffffu) + bf16_to_f32(lw[q] & 0xffffu);
                        const float h1 = __uint_as_float(hw[q] & 0xffff0000u) + __uint_as_float(lw[q] & 0xffff0000u);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t w = q == 0 ? bv[e].x : q == 1 ? bv[e].y : q == 2 ? bv[e].z : bv[e].w;
                            low[e] += h0 * bf16_to_f32(w & 0xffffu) + h1 * __uint_as_float(w & 0xffff0000u);
                        }
                    }
                }
            }
        }
        float v[4];
        sum_parts(parts, M * N, split, m * N + n, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += low[e];
        const int64_t to = lr.order ? lr.order[m] : m;
        *reinterpret_cast<uint2*>(c + to * N + n) = pack4_bf16(v);
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
        sum_parts(parts, M * N, split, row * N + n, v);
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

// Rows block, block + blocks, .. of out = bf16(r[row] x), a row's 16-byte pieces by thread.
struct ScaleRows {
    const uint16_t* x;
    const float* r;
    int64_t M;
    int C8;                // row length in eights
    uint16_t* out;
};
__device__ __forceinline__ void scale_rows(const ScaleRows& s, int block, int blocks) {
    for (int64_t row = block; row < s.M; row += blocks) {
        const float sc = s.r[row];
        for (int c = threadIdx.x; c < s.C8; c += 256) {
            const int64_t i = row * s.C8 + c;
            const uint4 v = *reinterpret_cast<const uint4*>(s.x + i * 8);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            float f[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[2 * e] = bf16_to_f32(w[e] & 0xffffu) * sc;
                f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u) * sc;
            }
            *reinterpret_cast<uint4*>(s.out + i * 8) = pack8(f);
        }
    }
}
__global__ void __launch_bounds__(256)
scale_rows_kernel(ScaleRows s) {
    scale_rows(s, (int)blockIdx.x, (int)gridDim.x);
}

// Gradients' work that does not depend on each other, in one launch: the data gradient's
// tiles (all, or what the large kernel left), the weight gradient's, the scaled copy of an
// operand, dr of an earlier launch's partial sums.  A small call's workgroups fill the GPU
// together, and a launch costs 2 to 3 us on the host as on the GPU.
struct GradJobs {
    SmallArgs d, w;
    ScaleRows s;
    const float* drp;
    float* dr;
    int64_t dr_rows;
    int dr_parts;
    int nd, nw, ns, nr;    // workgroups of each (nd, nw multiples of 128)
};
// MB and ST are the data gradient's.
template <int MB, int ST>
__global__ void __launch_bounds__(256, per_cu(MB, ST))
bf16_grad_kernel(GradJobs j) {
    constexpr bool with_w = per_cu(MB, ST) == 2;    // (weight gradients always share CUs)
    union Smem {
        uint8_t d[ST][small_stage(MB)], w[with_w ? 2 : 1][small_stage(2)];
    };
    __shared__ __attribute__((aligned(16))) Smem sm;
    int b = (int)blockIdx.x;
    if (b < j.nd) return small_tile<Bf16Form::kDataGrad, MB, ST>(j.d, b, sm.d);
    b -= j.nd;
    if constexpr (with_w) {
        if (b < j.nw) return small_tile<Bf16Form::kWeightGrad, 2, 2>(j.w, b, sm.w);
        b -= j.nw;
    }
    if (b < j.ns) return scale_rows(j.s, b, j.ns);
    b -= j.ns;
    const int64_t row = (int64_t)b * 256 + threadIdx.x;
    if (row < j.dr_rows) {
        float sum = 0.f;
#pragma unroll 16
        for (int i = 0; i < j.dr_parts; ++i) sum += j.drp[i * j.dr_rows + row];
        j.dr[row] = sum;
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of a call (an upper bound where groups own rows: their counts are on the device).
int64_t small_tiles(const Bf16Problem& p, int MB) {
    const int64_t ntn = cdiv(p.N, SM_N), bm = small_m(MB);
    if (p.form == Bf16Form::kForward) return cdiv(p.M, bm) * ntn;
    if (p.form == Bf16Form::kDataGrad || p.form == Bf16Form::kDown)     // sum of ceil(rows / bm) <= this
        return (p.rows < p.G ? p.rows : p.G + (p.rows - p.G) / bm) * ntn;
    return (int64_t)p.G * cdiv(p.M, bm) * ntn;
}

// ---- which kernel ------------------------------------------------------------------
enum Kind { kLarge = 0, kSmall = 1, kMiddle = 2 };     // (kSmall, kMiddle: also MB)
struct Plan {
    Kind kind;
    int split;
    bool alone = false;    // middle tiles, at most one workgroup a CU: four stages
};

// Rows of groups are on the device: groups are taken as equal here.
//
// Products whose groups own rows: the fastest by a model of their times, in us, its
// numbers measured at K x N of 4096 x 4096, 1408 x 2064, 4096 x 14336, 14336 x 4096 and
// 1024 x 1024 with 17 to 8192 rows, and at 1 to 64 experts with 4 to 4096 rows each.  A
// tile's step of 64 in K takes a CU 0.31 (small) or 0.48 (middle) for a workgroup alone, 0.30
// or 0.47 a workgroup when it has several, and 1.6 (large, four middle ones' work); starting
// and storing take 6, a large round 12 in all; adding the shares of a split K takes 4.5 and
// the time its bytes need.  A last round of large tiles goes to middle ones where
// whole_rounds says so.  The adapters' down projection of few rows takes half of the CUs
// beside the tiles of a split K (K x N = 14336 x 4096, 128 rows, middle tiles: 256 of them 59
// us, 128 37), or a launch of its own of K / 512.
Plan plan_rows(const Bf16Problem& p) {
    const int64_t groups = p.form == Bf16Form::kForward ? 1 : p.rows < p.G ? p.rows : p.G;
    const int64_t rows = groups ? cdiv(p.rows, groups) : 0;
    const double nk = (double)cdiv(p.K, SM_K);
    auto tiles = [&](int bm, int bn) { return (double)(groups * cdiv(rows, bm) * cdiv(p.N, bn)); };
    const bool beside = p.form == Bf16Form::kForward && p.rows <= kLoraUnsorted && few_low_rank(p.rows, p.N, p.lr.r);
    auto tile_us = [&](Kind k, double units, double steps, double cus) {
        const double each = units / cus, most = units <= 2 * cus ? 2 : (double)(((int64_t)units - 1) / (int64_t)cus + 1);
        if (k == kSmall) return steps * (each <= 1 ? 0.31 : 0.30 * most);
        return steps * (each <= 1 ? 0.48 : each <= 2 ? 0.37 + 0.27 * each : 0.47 * most);
    };
    Plan best{kSmall, 1};
    double least = 1e30;
    for (Kind k : {kSmall, kMiddle}) {
        const double t = tiles(small_m(k), SM_N);
        // Sums of one to three steps are starting and storing, half as long for a small tile:
        // middle ones only where small ones take a second round (us, small and middle: x w^T
        // of 456 rows, K x N = 64 x 4176 10.4 and 12.2, 4096 rows, 128 x 4096 24.9 and 22.3)
        if (k == kMiddle && nk < 4 && tiles(small_m(kSmall), SM_N) <= 512) continue;
        // (a share keeps four steps)
        for (int split = 1; split == 1 || (split <= 16 && nk >= 4.0 * split && t * split <= 1024); ++split) {
            double us = 6 + tile_us(k, t * split, nk / split, beside && split > 1 ? 128 : 256);
            if (beside && split == 1) us += p.K / 512;
            if (split > 1) us += 4.5 + 8e-6 * split * p.rows * p.N / 3;
            if (us < least) {
                least = us;
                best = Plan{k, split, small_tiles(p, k) * split <= 256};
            }
        }
    }
    const double t = tiles(256, 256);
    if (t < 1e9) {
        const int whole = whole_rounds((int)t, 256), rest = (int)t - whole;
        const double us = cdiv(whole, 256) * 1.6 * nk + (whole ? 12 : 0) + (rest ? 6 + tile_us(kMiddle, 4.0 * rest, nk, 256) : 0);
        if (whole && us < least) best = Plan{kLarge, 1, rest > 0 && rest <= 64};      // (alone: the rest)
    } else {
        best = Plan{kLarge, 1, false};
    }
    return best;
}

// Weight gradients: the large tiles' chains hide the stores that take most of the time
// where groups have few rows, but a few rounds of them wait for the group with most rows
// (8 experts of 2816 x 1024, 16384 rows falling as 1 / rank^1.1: 165 us, middle tiles
// 122; even: 109 and 111).  One group has no such thing, only a last round partly used
// (4096 x 4096, 2048 rows: 59 us, middle 75).  Middle tiles split long sums where there
// are few (8 of 512 x 512, 16384 rows: 27 us, large 52).  How many shares goes by groups of
// equal rows: one group with all of them keeps a long sum (81 us there, even 22).
Plan plan_weights(const Bf16Problem& p) {
    const int64_t large = p.G * cdiv(p.M, 256) * cdiv(p.N, 256);
    const int64_t last = large % 256;
    if (large >= 1024 || (p.G == 1 && large >= 192 && (last == 0 || last >= 192))) return Plan{kLarge, 1};
    const int64_t tiles = p.G * cdiv(p.M, small_m(kMiddle)) * cdiv(p.N, SM_N);
    const int64_t nk = cdiv(cdiv(p.rows, p.G), SM_K);
    // a share keeps 16 steps
    int64_t split = 512 / tiles;
    if (split > nk / 16) split = nk / 16;
    return Plan{kMiddle, split < 1 ? 1 : split > 16 ? 16 : (int)split};
}

Plan plan_of(const Bf16Problem& p) {
    return p.form == Bf16Form::kWeightGrad ? plan_weights(p) : plan_rows(p);
}

// Workgroups of the small or middle tiles of a call.
int64_t small_grid(const Bf16Problem& p, const Plan& q) { return cdiv(small_tiles(p, q.kind) * q.split, 128) * 128; }

}  // namespace

int64_t bf16_parts(const Bf16Problem& p) {
    const Plan q = plan_of(p);
    return q.split > 1 ? q.split * (p.form == Bf16Form::kWeightGrad ? (int64_t)p.G * p.M : p.rows) * p.N : 0;
}

int64_t bf16_product_tiles(const Bf16Problem& p) {
    const Plan q = plan_of(p);
    return q.kind == kLarge ? small_tiles(p, kMiddle) / 128 : small_grid(p, q);
}

int64_t bf16_dr_parts(int64_t N) { return cdiv(N, 64); }

extern "C" int32_t mx_internal_bf16_plan(int32_t form, int32_t G, int64_t rows, int64_t M, int64_t N, int64_t K,
                                         int32_t r) {
    Bf16Problem p{};
    p.form = (Bf16Form)form;
    p.G = G;
    p.rows = rows;
    p.M = M; p.N = N; p.K = K;
    p.lr.r = r;
    const Plan q = plan_of(p);
    return q.kind + 4 * q.split;
}

namespace {

// Workgroups of the middle tiles that take what the large kernel left, where only the
// device knows how much.
constexpr int kRestGrid = (4 * kTailMost + 127) / 128 * 128;

hipError_t join_shares(const Bf16Problem& p, int split, hipStream_t st) {
    const int64_t all = (p.form == Bf16Form::kWeightGrad ? (int64_t)p.G * p.M : p.rows) * p.N;
    if (p.rscale)
        hipLaunchKernelGGL(bf16_join_rows_kernel, dim3((unsigned)p.M), dim3(256), 0, st, p.parts, p.M, p.N, split,
                           p.rscale, p.drx, static_cast<uint16_t*>(p.C), p.dr);
    else
        hipLaunchKernelGGL(bf16_join_kernel, dim3((unsigned)cdiv(all, 1024)), dim3(256), 0, st, p.parts, all, split,
                           p.C, p.c_f32, p.c_add);
    return hipGetLastError();
}

// d: the data gradient's plan (its tiles, or what the large kernel leaves).
hipError_t launch_jobs(GradJobs& j, const Plan& d, hipStream_t st) {
    const int grid = j.nd + j.nw + j.ns + j.nr;
    if (grid == 0) return hipSuccess;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, st, j); };
    if (j.nd && d.kind == kSmall) go(bf16_grad_kernel<1, 3>);
    else if (j.nd && !j.nw && d.alone) go(bf16_grad_kernel<2, 4>);
    else go(bf16_grad_kernel<2, 2>);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_down_tiles(const LoraDown& d, hipStream_t st) {
    Bf16Problem p{};
    p.form = Bf16Form::kDown;
    p.G = d.L;
    p.rows = d.M;
    p.M = d.M; p.N = d.r; p.K = d.K;
    p.offs = d.offs;
    p.A = d.x;
    p.B = d.a;
    p.C = d.h;
    p.rscale = d.scale;
    p.lr.order = d.order;
    const unsigned grid = (unsigned)(cdiv(small_tiles(p, 1), 128) * 128);
    hipLaunchKernelGGL(bf16_down_kernel, dim3(grid), dim3(256), 0, st, SmallArgs{p, 1, false, 0});
    return hipGetLastError();
}

hipError_t launch_lora_product(const Bf16Problem& p, const LoraDown& d, hipStream_t st) {
    const Plan q = plan_of(p);
    const dim3 bd(256);
    // The join adds the adapters' part where that is small, and twice that much for unsorted
    // rows of many adapters in more than two shares (72 rows, 4096 x 4096, rank 128, us: 16
    // adapters 74 in the tiles, 50 in the join, 64 adapters 115 and 58; 4 adapters 39 and 45; two
    // shares of 64 rows, 4096 x 14336, rank 64, 16 adapters 56 and 87).
    const bool join_lr = q.split > 1 && (few_low_rank(p.M, p.N, p.lr.r) ||
                                         (q.split > 2 && !d.order && d.L > 4 &&
                                          p.M * p.N * p.lr.r <= 2 * kFewLowRank));
    // then h can be made beside the tiles
    const bool with_down = join_lr && !d.order && p.M * d.r <= kDownFine;
    hipError_t e = with_down ? hipSuccess : launch_lora_down(d, st);
    if (e != hipSuccess) return e;
    if (q.kind == kLarge) {
        e = launch_bf16_large(p, true, st);
        if (e != hipSuccess) return e;
        const int grid = bf16_large_grid(), all = (int)(cdiv(p.M, 256) * cdiv(p.N, 256));
        const int left = (int)cdiv((all - whole_rounds(all, grid)) * 4, 128) * 128;
        if (left == 0) return hipSuccess;
        const SmallArgs rest{p, 1, true, grid};
        auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(left), bd, 0, st, rest); };
        q.alone ? go(bf16_forward_kernel<2, 4>) : go(bf16_forward_kernel<2, 2>);
        return hipGetLastError();
    }
    const SmallArgs a{p, q.split, !join_lr, 0};
    const int tiles = (int)small_grid(p, q);
    if (with_down) {
        const dim3 gd((unsigned)(tiles + cdiv(p.M, 16) * d.r));
        auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, gd, bd, 0, st, a, d, tiles); };
        if (q.kind == kSmall) go(bf16_forward_down_kernel<1, 3>);
        else q.alone ? go(bf16_forward_down_kernel<2, 4>) : go(bf16_forward_down_kernel<2, 2>);
    } else {
        auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(tiles), bd, 0, st, a); };
        if (q.kind == kSmall) go(bf16_forward_kernel<1, 3>);
        else q.alone ? go(bf16_forward_kernel<2, 4>) : go(bf16_forward_kernel<2, 2>);
    }
    e = hipGetLastError();
    if (e != hipSuccess || q.split == 1) return e;
    const dim3 gj((unsigned)cdiv(p.N, 1024), (unsigned)(p.M < 65535 ? p.M : 65535));
    auto join = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, gj, bd, 0, st, p.parts, p.M, p.N, q.split, p.lr, static_cast<uint16_t*>(p.C));
    };
    join_lr ? join(bf16_join_adapters_kernel<true>) : join(bf16_join_adapters_kernel<false>);
    return hipGetLastError();
}

hipError_t launch_linear_grads(const Bf16Problem* d, const Bf16Problem* w, const uint16_t* scale_x,
                               const float* scale_r, int64_t scale_cols, uint16_t* scaled, hipStream_t st) {
    const Plan pd = d ? plan_of(*d) : Plan{kLarge, 1}, pw = w ? plan_of(*w) : Plan{kLarge, 1};
    const bool d_tiles = d && pd.kind != kLarge, w_tiles = w && pw.kind != kLarge;
    bool dr_left = d && d->drp && !(d_tiles && pd.split > 1);    // (the rows' join makes dr)
    const ScaleRows sr{scale_x, scale_r, w ? w->rows : 0, (int)(scale_cols / 8), scaled};
    // a scaled copy goes with the data gradient's tiles if it is small, else before them
    const bool scale_with = scaled && d_tiles && sr.M * scale_cols <= (int64_t)1 << 22;
    hipError_t e = hipSuccess;
    if (scaled && !scale_with) {
        hipLaunchKernelGGL(scale_rows_kernel, dim3((unsigned)(sr.M < 65536 ? sr.M : 65536)), dim3(256), 0, st, sr);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (d && !d_tiles) {
        e = launch_bf16_large(*d, true, st);
        if (e != hipSuccess) return e;
    }
    GradJobs j{};
    if (d) {
        j.d = d_tiles ? SmallArgs{*d, pd.split, false, 0} : SmallArgs{*d, 1, false, bf16_large_grid()};
        j.nd = d_tiles ? (int)small_grid(*d, pd) : kRestGrid;
    }
    auto with_w = [&] {
        j.w = SmallArgs{*w, pw.split, false, 0};
        j.nw = (int)small_grid(*w, pw);
    };
    const bool w_now = w_tiles && !scale_with;
    if (w_now) with_w();
    if (scale_with) {
        j.s = sr;
        j.ns = (int)(sr.M < 512 ? sr.M : 512);
    }
    e = launch_jobs(j, pd, st);
    if (e == hipSuccess && d_tiles && pd.split > 1) e = join_shares(*d, pd.split, st);
    if (e != hipSuccess) return e;
    GradJobs k{};
    if (w_tiles && !w_now) {
        j = k;
        with_w();
        k = j;
    }
    if (dr_left) {
        k.drp = d->drp;
        k.dr = d->dr;
        k.dr_rows = d->M;
        k.dr_parts = (int)bf16_dr_parts(d->N);
        k.nr = (int)cdiv(d->M, 256);
    }
    e = launch_jobs(k, pd, st);
    if (e == hipSuccess && w && !w_tiles) e = launch_bf16_large(*w, false, st);
    if (e == hipSuccess && w_tiles && pw.split > 1) e = join_shares(*w, pw.split, st);
    return e;
}

}  // namespace mx
