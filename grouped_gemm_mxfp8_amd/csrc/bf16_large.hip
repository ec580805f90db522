// bf16 products in 256 x 256 tiles (gfx950): the data and weight gradients of
// GroupedLinear and the adapter linear, for calls with enough of them.
//
// One persistent workgroup of four waves per CU, each wave 128 x 128 of a tile (4 x 4
// accumulators of the 32x32x16 MFMA, all 256 AGPRs).  K goes in steps of 64 through
// two LDS stages of 64 KB filled by direct loads; a step is 64 MFMAs of 32 cycles, and
// the 16 loads and the next step's fragment reads are issued one by one in their
// shadow.  A workgroup's tiles form a chain: the last two steps of a tile load the
// next tile's first two, and its output leaves from the registers while they land.
//
// Fragments of a step are in registers before it begins, so its stage can be refilled
// during the step.  First pass (rows 0, 1 of the wave's blocks), with most loads of
// step + 2; then the loads of step + 1 have landed, and the second pass (rows 2, 3)
// reads the next fragments into the registers its MFMAs free.
//
// LDS orders as in the small tiles (bf16_small.hip): along K, 128-byte lines with chunk
// c of line n at c ^ (n >> 1 & 7); across K, 512-byte rows with 64-byte pieces at
// piece ^ (k & 3).
#include "bf16_tiles.h"

namespace mx {
namespace {

constexpr int BM = 256, BN = 256, BK = 64, NT = 256;
constexpr int STAGE = 256 * 128;                   // bytes of an operand's step
constexpr int LOADS = 16, FIRST = 10;              // per wave and step; in the first pass

// Slot of a pass after which load u of n is issued, over slots [first, first + span).
constexpr int slot_of(int u, int n, int first, int span) { return first + (2 * u + 1) * span / (2 * n); }
constexpr int load_first(int t) {                  // the loads follow the barrier after slot 3
    for (int u = 0; u < FIRST; ++u)
        if (slot_of(u, FIRST, 4, 28) == t) return u;
    return -1;
}
constexpr int load_second(int t) {
    for (int u = 0; u < LOADS - FIRST; ++u)
        if (slot_of(u, LOADS - FIRST, 8, 16) == t) return FIRST + u;
    return -1;
}
constexpr bool loads_covered() {
    int n = 0;
    for (int t = 0; t < 32; ++t) n += (load_first(t) >= 0) + (load_second(t) >= 0);
    return n == LOADS;
}
static_assert(loads_covered(), "every load has a slot of its own");

struct Tile {
    int g;
    int64_t m0, mvalid, n0;
};
// Operands of a tile: base addresses, bytes from there to the end of what belongs to
// the tile's group, K steps.
struct Src {
    const uint8_t *a, *b;
    int64_t an, bn;
    int nk;
};

// TAIL: K % 64 != 0 of an operand along K.  OUT: what is stored.
enum class Out { kBf16, kScaled, kAdapters, kF32, kAdd };

template <Bf16Form F, bool TAIL, Out OUT>
__global__ void __launch_bounds__(NT, 1)
bf16_large_kernel(Bf16Problem p, bool leave_tail) {
    constexpr bool kA = F != Bf16Form::kWeightGrad;       // A lies along K
    constexpr bool kB = F == Bf16Form::kForward;          // B lies along K
    constexpr bool kRows = F != Bf16Form::kWeightGrad;    // groups own rows of C
    struct Smem {
        uint8_t a[2][STAGE], b[2][STAGE];
    };
    __shared__ __attribute__((aligned(16))) Smem sm;
    __shared__ int s_prefix[kMaxGroups + 1];
    __shared__ int64_t s_offs[kMaxGroups + 1];
    __shared__ int s_order[kRows ? 1 : kMaxGroups];
    __shared__ float s_rsw[OUT == Out::kScaled ? 4 * 128 : 1];
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int G = p.G;
    const int ntn = (int)((p.N + BN - 1) / BN);
    const int ntm = (int)((p.M + BM - 1) / BM);           // of a group (not kDataGrad)

    // ---- tile table ----
    if constexpr (F != Bf16Form::kForward) {
        for (int g = tid; g <= G; g += NT) s_offs[g] = p.offs[g];
        __syncthreads();
    }
    if constexpr (F == Bf16Form::kDataGrad) {
        if (wave == 0) {
            int cnt[kMaxGroups / 64], local = 0;
#pragma unroll
            for (int u = 0; u < kMaxGroups / 64; ++u) {
                const int g = (tid & 63) * (kMaxGroups / 64) + u;
                int c = 0;
                if (g < G) {
                    const int64_t n = s_offs[g + 1] - s_offs[g];
                    c = n > 0 ? (int)((n + BM - 1) / BM) * ntn : 0;
                }
                cnt[u] = c;
                local += c;
            }
            int incl = local;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(incl, d);
                if ((tid & 63) >= d) incl += o;
            }
            int run = incl - local;
#pragma unroll
            for (int u = 0; u < kMaxGroups / 64; ++u) {
                const int g = (tid & 63) * (kMaxGroups / 64) + u;
                if (g < G) {
                    s_prefix[g] = run;
                    run += cnt[u];
                }
            }
            if (tid == 63) s_prefix[G] = incl;
        }
        __syncthreads();
    }
    if constexpr (!kRows) {
        // groups by falling rows, so that the longest sums begin first
        for (int g = tid; g < G; g += NT) {
            const int64_t n = s_offs[g + 1] - s_offs[g];
            int rank = 0;
            for (int o = 0; o < G; ++o) {
                const int64_t m = s_offs[o + 1] - s_offs[o];
                rank += m > n || (m == n && o < g);
            }
            s_order[rank] = g;
        }
        __syncthreads();
    }
    int total = F == Bf16Form::kDataGrad ? uni(s_prefix[G]) : (kRows ? 1 : G) * ntm * ntn;
    if (leave_tail) total = whole_rounds(total, gridDim.x);
    // workgroup b runs on XCD b % 8: each XCD takes a contiguous run of tiles a round
    const int grid = gridDim.x, bid = blockIdx.x;
    const int slot = (grid % 8 == 0) ? (bid % 8) * (grid / 8) + bid / 8 : bid;

    auto locate = [&](int t) -> Tile {
        int g = 0, local = t, mtiles = ntm;
        int64_t base = 0, rows = p.M;
        if constexpr (F == Bf16Form::kDataGrad) {
            int lo = 0, hi = G - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_prefix[mid] <= t) lo = mid; else hi = mid - 1;
            }
            g = lo;
            local = t - s_prefix[g];
            mtiles = (s_prefix[g + 1] - s_prefix[g]) / ntn;
            base = s_offs[g];
            rows = s_offs[g + 1] - base;
        } else if constexpr (!kRows) {
            const int o = t / (ntm * ntn);
            local = t - o * (ntm * ntn);
            g = s_order[o];
        }
        const TileAt at = band_order(local, mtiles, ntn);
        const int64_t m = (int64_t)at.m * BM;
        return Tile{uni(g), uni64(base + m), uni64(min((int64_t)BM, rows - m)), uni64((int64_t)at.n * BN)};
    };
    const int64_t lda = kA ? p.K : p.M, ldb = kB ? p.K : p.N;
    // bytes a step moves an operand's base by (along K the step is part of the offset)
    const int64_t astep = kA ? 0 : BK * lda * 2, bstep = kB ? 0 : BK * ldb * 2;
    const int nk_all = (int)((p.K + BK - 1) / BK);
    auto src_of = [&](const Tile& t) -> Src {
        Src s;
        const uint16_t *a = p.A, *b = p.B;
        s.nk = nk_all;
        if constexpr (F == Bf16Form::kWeightGrad) {
            const int64_t row0 = uni64(s_offs[t.g]);
            const int64_t rows = max((int64_t)0, uni64(s_offs[t.g + 1]) - row0);
            s.nk = (int)((rows + BK - 1) / BK);
            s.a = reinterpret_cast<const uint8_t*>(a + row0 * lda + t.m0);
            s.an = (rows * lda - t.m0) * 2;
            s.b = reinterpret_cast<const uint8_t*>(b + row0 * ldb + t.n0);
            s.bn = (rows * ldb - t.n0) * 2;
        } else {
            s.a = reinterpret_cast<const uint8_t*>(a + t.m0 * lda);
            s.an = t.mvalid * lda * 2;
            if (F == Bf16Form::kForward && p.lr.order) {
                s.a = reinterpret_cast<const uint8_t*>(a);
                s.an = p.M * lda * 2;
            }
            if constexpr (F == Bf16Form::kDataGrad) {
                s.b = reinterpret_cast<const uint8_t*>(b + (int64_t)t.g * p.K * p.N + t.n0);
                s.bn = (p.K * p.N - t.n0) * 2;
            } else {
                s.b = reinterpret_cast<const uint8_t*>(b + t.n0 * ldb);
                s.bn = min((int64_t)BN, p.N - t.n0) * ldb * 2;
            }
        }
        return s;
    };

    if (slot < total) {
        const uint32_t smb = (uint32_t)uni((int)lds_addr(&sm));
        int w = slot;
        Tile L = locate(w);
        bool pre = false;
        int base = 0;          // stage of the tile's step 0
        // (rows of A in another order: each load's own offsets, kept for the whole tile and
        // set to the next one's when its loads begin; a row past the last loads nothing)
        constexpr bool kOrder = OUT == Out::kAdapters;
        uint32_t ro[kOrder ? 8 : 1];
        auto rows_of = [&](const Tile& t) {
            if constexpr (kOrder) {
                const int ln = lane_now();
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int row = wave * 64 + u * 8 + (ln >> 3);
                    const int64_t from = !p.lr.order ? row : row < t.mvalid ? p.lr.order[t.m0 + row] : -1;
                    ro[u] = (from < 0 ? 0x80000000u : (uint32_t)(from * lda * 2)) +
                            (uint32_t)(((ln & 7) ^ (ln >> 4)) ^ (u & 1 ? 4 : 0)) * 16u;
                }
            }
        };
        rows_of(L);
        for (;;) {
            const int wnext = w + grid;
            const bool has_next = wnext < total;
            const int lane = lane_now();
            const int l32 = lane & 31, half = lane >> 5;
            const Src own = src_of(L);
            const int nk = own.nk;

            // ---- direct loads: a lane's offsets, and how odd loads differ ----
            // along K: 8 rows a load, lane l row l >> 3 and the chunk stored at l & 7;
            // across K: 2 rows a load, lane l row l >> 5, the chunk stored at l & 31
            auto offset = [&](bool along, int64_t ld, uint32_t& off, uint32_t& flip) {
                if (along) {
                    const int c = (lane & 7) ^ (lane >> 4);
                    off = (uint32_t)((wave * 64 + (lane >> 3)) * ld * 2) + (uint32_t)c * 16u;
                    flip = (c & 4) ? (uint32_t)-64 : 64u;
                } else {
                    const int c = (lane & 31) ^ (half << 2);
                    off = (uint32_t)((wave * 16 + half) * ld * 2) + (uint32_t)c * 16u;
                    flip = (c & 8) ? (uint32_t)-128 : 128u;
                }
            };
            uint32_t aoff, aflip, boff, bflip;
            offset(kA, lda, aoff, aflip);
            offset(kB, ldb, boff, bflip);
            // (TAIL) the lanes whose chunk of the last step lies past K, for even and odd loads
            const int tail = (int)(p.K - (int64_t)(nk_all - 1) * BK);
            const int tc = (lane & 7) ^ (lane >> 4);
            const uint32_t over0 = TAIL && tc * 8 >= tail ? 0x80000000u : 0u;
            const uint32_t over1 = TAIL && (tc ^ 4) * 8 >= tail ? 0x80000000u : 0u;
            struct Rsrc {
                v4i a, b;
                uint32_t soff, o0, o1;
            };
            // descriptors of step ks of s; LIVE: ks < nk is known
            auto rsrc_of = [&](const Src& s, int ks, auto livec) -> Rsrc {
                const bool live = decltype(livec)::value || ks < s.nk;
                const bool last = TAIL && ks + 1 == nk_all;
                return Rsrc{make_rsrc(s.a + ks * astep, live ? s.an - ks * astep : 0),
                            make_rsrc(s.b + ks * bstep, live ? s.bn - ks * bstep : 0), (uint32_t)ks * 128u,
                            last ? over0 : 0u, last ? over1 : 0u};
            };
            auto dma = [&](auto uc, const Rsrc& r, int st) {
                constexpr int u = decltype(uc)::value;
                if constexpr (u < 8) {
                    uint32_t off;
                    if constexpr (kOrder) off = ro[u];
                    else off = aoff + (uint32_t)(u * (kA ? 8 : 2) * lda * 2) + (u & 1 ? aflip : 0u);
                    dma_b128<u * 1024>(r.a, smb + (uint32_t)offsetof(Smem, a) + st * STAGE + wave * 8192,
                                       TAIL && kA ? off | (u & 1 ? r.o1 : r.o0) : off, kA ? r.soff : 0u);
                } else {
                    constexpr int v = u - 8;
                    const uint32_t off = boff + (uint32_t)(v * (kB ? 8 : 2) * ldb * 2) + (v & 1 ? bflip : 0u);
                    dma_b128<v * 1024>(r.b, smb + (uint32_t)offsetof(Smem, b) + st * STAGE + wave * 8192,
                                       TAIL && kB ? off | (v & 1 ? r.o1 : r.o0) : off, kB ? r.soff : 0u);
                }
            };

            // ---- fragments ----
            bf16x8 af[4][4], bf[4][4];             // block, sixteen of K
            const int swz = (l32 >> 1) & 7;
            // along: the line of block 0 and its chunk of each sixteen; across: row
            // (l >> 2) & 3 of eight half and the lane's 8 bytes of each block's piece
            const int a_line = (wm * 128 + l32) * 128, b_line = (wn * 128 + l32) * 128;
            const int t_row = (8 * half + ((lane >> 2) & 3)) * 512, t_piece = (lane >> 2) & 3;
            const int t_in = 32 * ((lane >> 4) & 1) + 8 * (lane & 3);
            auto read = [&](bool along, const uint8_t* st, int line, int wpart, int i, int s) -> bf16x8 {
                if (along) return frag_along(st + line + i * 4096 + (((2 * s + half) ^ swz) << 4));
                return frag_across(st + t_row + s * 8192 + (((wpart * 4 + i) ^ t_piece) << 6) + t_in, 2048);
            };
            auto read_a = [&](auto ic, auto sc, int st) {
                constexpr int i = decltype(ic)::value, s = decltype(sc)::value;
                af[i][s] = read(kA, sm.a[st], a_line, wm, i, s);
            };
            auto read_b = [&](auto jc, auto sc, int st) {
                constexpr int j = decltype(jc)::value, s = decltype(sc)::value;
                bf[j][s] = read(kB, sm.b[st], b_line, wn, j, s);
            };
            v16f acc[4][4];
            // Slot t of a pass over rows i0, i0 + 1: column t / 8, sixteen t / 2 % 4 of K, row
            // i0 + t % 2 (an MFMA that follows the one whose result it adds to would wait).
            // FIRSTK: the sums start from zero.
            auto mfma = [&](auto tc_, auto i0c, auto firstc) {
                constexpr int t = decltype(tc_)::value, j = t / 8, s = t / 2 % 4, i = decltype(i0c)::value + t % 2;
                const v16f c = decltype(firstc)::value && s == 0 ? zero16() : acc[i][j];
                acc[i][j] = mfma_bf16(bf[j][s], af[i][s], c);
            };
            auto step = [&](int ks, const Src& s, int kl, auto livec, auto firstc) {
                const int cur = (base + ks) & 1, nxt = cur ^ 1;
                const Rsrc r = rsrc_of(s, kl, livec);
                static_for<32>([&](auto tc_) {
                    constexpr int t = decltype(tc_)::value;
                    // every wave holds this step's fragments: the stage is free
                    if constexpr (t == 4) lds_barrier();
                    mfma(tc_, std::integral_constant<int, 0>{}, firstc);
                    __builtin_amdgcn_sched_barrier(0);
                    constexpr int u = load_first(t);
                    if constexpr (u >= 0) dma(std::integral_constant<int, u>{}, r, cur);
                    __builtin_amdgcn_sched_barrier(0);
                });
                wait_vm<FIRST>();          // this wave's loads of step ks + 1 have landed
                lds_barrier();             // and everybody's
                static_for<32>([&](auto tc_) {
                    constexpr int t = decltype(tc_)::value, j = t / 8, q = t % 8;
                    mfma(tc_, std::integral_constant<int, 2>{}, firstc);
                    __builtin_amdgcn_sched_barrier(0);
                    if constexpr (t < 8)
                        read_a(std::integral_constant<int, t % 2>{}, std::integral_constant<int, t / 2>{}, nxt);
                    if constexpr (j > 0 && q < 4)
                        read_b(std::integral_constant<int, j - 1>{}, std::integral_constant<int, q>{}, nxt);
                    // in the last column a sixteen's fragments are free after its MFMAs
                    if constexpr (t >= 24 && t % 2 == 1) {
                        constexpr int k = (t - 24) / 2;
                        read_a(std::integral_constant<int, 2>{}, std::integral_constant<int, k>{}, nxt);
                        read_a(std::integral_constant<int, 3>{}, std::integral_constant<int, k>{}, nxt);
                        read_b(std::integral_constant<int, 3>{}, std::integral_constant<int, k>{}, nxt);
                    }
                    constexpr int u = load_second(t);
                    if constexpr (u >= 0) dma(std::integral_constant<int, u>{}, r, cur);
                    __builtin_amdgcn_sched_barrier(0);
                });
            };

            if (!pre) {
                wait_vm<0>();
                lds_barrier();                     // no load in flight, stages free
            }
            if constexpr (OUT == Out::kScaled) {
                // the wave's 128 row scales (rows past the tile read 0); the previous
                // tile's epilogue has read its own
                const int64_t n = min((int64_t)128, max((int64_t)0, L.mvalid - wm * 128));
                const v4i rr = make_rsrc(p.rscale + L.m0 + wm * 128, n * 4);
                const uint32_t la = (uint32_t)uni((int)lds_addr(&s_rsw[wave * 128]));
                dma_b32(rr, la, (uint32_t)lane * 4u, 0u);
                dma_b32(rr, la + 256u, (uint32_t)lane * 4u + 256u, 0u);
            }
            if (!pre) {
                const Rsrc r0 = rsrc_of(own, 0, std::false_type{}), r1 = rsrc_of(own, 1, std::false_type{});
                static_for<LOADS>([&](auto uc) { dma(uc, r0, base); });
                static_for<LOADS>([&](auto uc) { dma(uc, r1, base ^ 1); });
                wait_vm<LOADS>();
                lds_barrier();
            }
            static_for<4>([&](auto ic) {
                static_for<4>([&](auto sc) {
                    read_a(ic, sc, base);
                    read_b(ic, sc, base);
                });
            });
            int ks = 0;
            if (nk >= 3) {
                step(0, own, 2, std::true_type{}, std::true_type{});
                ks = 1;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = zero16();
            }
            for (; ks + 2 < nk; ++ks) step(ks, own, ks + 2, std::true_type{}, std::false_type{});
            Tile Ln = L;
            Src nx = own;
            nx.nk = 0;                             // no next tile: loads of no bytes
            if (has_next) {
                Ln = locate(wnext);
                nx = src_of(Ln);
                if (kOrder && p.lr.order) rows_of(Ln);    // (the tile's own loads are all issued)
            }
            for (; ks < nk; ++ks) step(ks, nx, ks + 2 - nk, std::false_type{}, std::false_type{});

            // ---- output ----
            {
                const int ln = lane_now();
                const int64_t rw = L.m0 + wm * 128, cw = L.n0 + wn * 128;
                const int rows = (int)(L.mvalid - wm * 128), cols = (int)min((int64_t)128, p.N - cw);
                const int64_t at = (kRows ? 0 : (int64_t)L.g * p.M * p.N) + rw * p.N + cw;
                int to[kOrder ? 4 : 1][4];
                if constexpr (kOrder) {
                    // all adapters' parts before the first store, whose completion the loads
                    // of the next part would wait for
#pragma unroll
                    for (int i = 0; i < 4; ++i) line_rows(to[i], p.lr.order, rw + 32 * i, rows - 32 * i, ln);
                    static_for<4>([&](auto ic) {
                        constexpr int i = decltype(ic)::value;
                        const int64_t row = rw + 32 * i + (ln & 31);
                        const bool there = (ln & 31) < rows - 32 * i;
                        int id = there ? p.lr.id[row] : -1;
                        if (id >= p.lr.L) id = -1;
                        const uint16_t* const hr = there ? p.lr.h + row * (2 * p.lr.r) : nullptr;
                        // half the columns at a time: what one adapter adds needs registers
                        // of its own
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            v16f part[2] = {acc[i][2 * h], acc[i][2 * h + 1]};
                            add_adapters<2, 2>(part, p.lr, hr, id, p.N, cw + 64 * h, ln);
                            acc[i][2 * h] = part[0];
                            acc[i][2 * h + 1] = part[1];
                        }
                    });
                }
                static_for<4>([&](auto ic) {
                    constexpr int i = decltype(ic)::value;
                    const int r0 = rows - 32 * i;
                    // the accumulators stay in AGPRs until their row block is stored
#pragma unroll
                    for (int j = 0; j < 4; ++j) asm volatile("" : "+a"(acc[i][j]));
                    if constexpr (OUT == Out::kF32 || OUT == Out::kAdd) {
                        float* const c = static_cast<float*>(p.C) + at + 32 * i * p.N;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            store_f32_32x32<OUT == Out::kAdd>(acc[i][j], reinterpret_cast<uint8_t*>(c + 32 * j),
                                                              p.N * 4, r0, cols - 32 * j, ln);
                    } else {
                        const int64_t row = rw + 32 * i + (ln & 31);
                        const bool there = (ln & 31) < r0;
                        float sc = 1.f;
                        if constexpr (OUT == Out::kScaled) {
                            sc = s_rsw[wave * 128 + 32 * i + (ln & 31)];
                            if (p.drp) {
                                const uint16_t* const xr = there ? p.drx + row * p.N + cw : nullptr;
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    if (cols <= 64 * h) break;
                                    float sum = 0.f;
#pragma unroll
                                    for (int j = 2 * h; j < 2 * h + 2; ++j)
                                        sum += dot_32(acc[i][j], xr ? xr + 32 * j : nullptr, cols - 32 * j, ln);
                                    sum += __shfl_xor(sum, 32);
                                    if (there && ln < 32) p.drp[(cw / 64 + h) * p.M + row] = sum;
                                }
                            }
                        }
                        uint8_t* const c = reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.C) + at + 32 * i * p.N);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if constexpr (kOrder)
                                store_bf16_32x64<false, true>(
                                    acc[i][2 * h], acc[i][2 * h + 1], 1.f,
                                    reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.C) + cw + 64 * h),
                                    (uint32_t)p.N * 2u, r0, cols - 64 * h, ln, to[i]);
                            else store_bf16_32x64<OUT == Out::kScaled>(acc[i][2 * h], acc[i][2 * h + 1], sc, c + 128 * h,
                                                                  (uint32_t)p.N * 2u, r0, cols - 64 * h, ln);
                    }
                    // one row block at a time (read ahead, later blocks would spill)
                    __builtin_amdgcn_sched_barrier(0);
                });
            }
            if (!has_next) break;
            pre = nk >= 2;                         // a tile of one step loads nothing ahead
            base = uni(pre ? (base + nk) & 1 : 0);
            w = wnext;
            L = Ln;
        }
    }
    // no load may still be landing in LDS when the workgroup ends
    wait_vm<0>();
}

}  // namespace

int bf16_large_grid() {
    const int grid = device_cu_count();
    return grid < 8 ? 8 : grid / 8 * 8;
}

hipError_t launch_bf16_large(const Bf16Problem& p, bool leave_tail, hipStream_t s) {
    const bool tail = p.K % BK != 0;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(bf16_large_grid()), dim3(NT), 0, s, p, leave_tail); };
    switch (p.form) {
        case Bf16Form::kForward:
            tail ? go(bf16_large_kernel<Bf16Form::kForward, true, Out::kAdapters>)
                 : go(bf16_large_kernel<Bf16Form::kForward, false, Out::kAdapters>);
            break;
        case Bf16Form::kDataGrad:
            if (p.rscale)
                tail ? go(bf16_large_kernel<Bf16Form::kDataGrad, true, Out::kScaled>)
                     : go(bf16_large_kernel<Bf16Form::kDataGrad, false, Out::kScaled>);
            else
                tail ? go(bf16_large_kernel<Bf16Form::kDataGrad, true, Out::kBf16>)
                     : go(bf16_large_kernel<Bf16Form::kDataGrad, false, Out::kBf16>);
            break;
        default:
            if (!p.c_f32) go(bf16_large_kernel<Bf16Form::kWeightGrad, false, Out::kBf16>);
            else if (p.c_add) go(bf16_large_kernel<Bf16Form::kWeightGrad, false, Out::kAdd>);
            else go(bf16_large_kernel<Bf16Form::kWeightGrad, false, Out::kF32>);
    }
    return hipGetLastError();
}

}  // namespace mx
