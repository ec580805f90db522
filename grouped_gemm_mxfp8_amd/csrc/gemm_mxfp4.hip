// GroupedLinear on MXFP4 weights, tile kernel (gfx950): y = x w_e^T with x
// MXFP4 or MXFP8, on the block-scaled 16x16x128 MFMA.
//
// One persistent workgroup of four waves per CU, 256 x 256 output tiles, each
// wave 128 x 128 (8 x 8 MFMA blocks, 256 fp32 accumulators).  Operands go
// global -> LDS with direct loads into two stages, ranges of the buffer
// descriptors return zeros past an expert's last row, and a workgroup's tiles
// form a chain: the last two K steps of a tile load the next tile's first two,
// and its output leaves straight from the accumulators while they land.
//
// A K step moves one 128-byte line of each x row: 128 values of MXFP8, 256 of
// MXFP4 (two MFMAs deep, at half the cycles each, so a step of either format
// keeps the matrix cores busy for 2048 cycles per wave).  The weights' rows
// are 64 or 128 bytes of a step.
//
// The sums are fp32.  With MXFP8 x the MFMA first cuts the eight products of
// each run of eight K values to multiples of 2^-13 of their largest, as in every
// MXFP8 product of the library: a sum is off by less than 2^-10 of its terms'
// magnitudes (a model of the rule: 2e-5 in RMS), against the 2^-8 of the bf16
// result.
//
// LDS layout: 128-byte lines of eight 16-byte chunks, chunk c of line n stored
// at c ^ (n & 7), or for MXFP4 x at c ^ (n & 7) ^ (n >> 3 & 1).  A line is one
// row (two rows where a step has 64 bytes of a row).  A cycle of a fragment
// read serves 16 lanes, those of two neighbouring q with eight rows each (0-3
// and 12-15 of one, 4-11 of the other), over 64 banks: these orders put the 16
// chunks that each format's lanes take on different banks (0 conflicts
// counted; with the first order for MXFP4 x, 12 % of the kernel's cycles).
#include "gemm_device.h"

namespace mx {
namespace {

constexpr int BM = 256, BN = 256, NT4 = 256;
constexpr int BAND = 8;

// What a K step of x format XF4 (MXFP4) or not (MXFP8) is made of.
template <bool XF4>
struct Fmt {
    static constexpr int kBK = XF4 ? 256 : 128;          // values
    static constexpr int kSub = XF4 ? 2 : 1;             // MFMAs deep
    static constexpr int kWBytes = kBK / 2;              // bytes of a weight row
    static constexpr int kALoads = 8, kBLoads = kWBytes / 16;   // code loads per wave
    static constexpr int kCodeLoads = kALoads + kBLoads;
    // block scales of a row and step: kSub dwords.  Loaded a step at a time
    // (4 bytes a lane), or (WIN) 16 bytes of a row at a time, a window of kWin
    // steps: a load instruction then asks for its 64 rows' lines half or a
    // quarter as often, and those requests were as many as the codes'.
    static constexpr int kWin = 4 / kSub;
    // loads issued in a step's first pass (rows 0..3); the rest, the scales
    // among them, in the second
    static constexpr int kNA = XF4 ? 11 : 8;
};
template <bool XF4, bool WIN>
struct Loads {
    using F = Fmt<XF4>;
    static constexpr int kScale = WIN ? 1 : F::kSub;            // per wave and operand
    static constexpr int kAll = F::kCodeLoads + 2 * kScale;
};

template <bool XF4, bool WIN>
struct Smem {
    static constexpr int kSRow = WIN ? 16 : 4 * Fmt<XF4>::kSub;   // scale bytes kept of a row
    uint8_t a[2][BM * 128];
    uint8_t b[2][BN * Fmt<XF4>::kWBytes];
    uint8_t as[2][BM * kSRow];                 // by step, or by window
    uint8_t bs[2][BN * kSRow];
    uint8_t none[WIN ? 1024 : 16];             // where a load of no bytes writes its zeros
};

// Slot after which load u of a pass of n loads is issued, over slots
// [first, first + span) of the pass's 32.
constexpr int slot_of(int u, int n, int first, int span) { return first + (2 * u + 1) * span / (2 * n); }
template <bool XF4>
constexpr int load_at_a(int s) {
    for (int u = 0; u < Fmt<XF4>::kNA; ++u)
        if (slot_of(u, Fmt<XF4>::kNA, 0, 32) == s) return u;
    return -1;
}
// (the second pass reads the next step's fragments in its first and last slots)
template <bool XF4, bool WIN>
constexpr int load_at_b(int s) {
    constexpr int n = Loads<XF4, WIN>::kAll - Fmt<XF4>::kNA;
    for (int u = 0; u < n; ++u)
        if (slot_of(u, n, 4, 23) == s) return Fmt<XF4>::kNA + u;
    return -1;
}
template <bool XF4, bool WIN>
constexpr bool loads_covered() {
    int n = 0;
    for (int s = 0; s < 32; ++s) n += (load_at_a<XF4>(s) >= 0) + (load_at_b<XF4, WIN>(s) >= 0);
    return n == Loads<XF4, WIN>::kAll && Fmt<XF4>::kNA <= Fmt<XF4>::kCodeLoads;
}
static_assert(loads_covered<true, true>() && loads_covered<false, true>() && loads_covered<true, false>() &&
                  loads_covered<false, false>(),
              "every load has a slot of its own, the scales' in the second pass");

template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Buffer descriptors of one tile and its K steps (0: no tile).
struct Src {
    v4i ra, rb, rsa, rsb;
    int nk;
};

struct Loc {
    int g;
    int64_t m0, mvalid, n0;
};

// HALF: K % 256 == 128 (MXFP4): the last step holds 128 values; its chunks 4..7
// are read past the descriptors' ranges, as zeros, and their scales as 0.
// WIN: scales in windows of 16 bytes, K >= 512 (a row has 16 of them).
// SCALED: row scales.
template <bool XF4, bool HALF, bool WIN, bool SCALED>
__global__ void __launch_bounds__(NT4, 1)
linear4_tile_kernel(GemmProblem p) {
    using F = Fmt<XF4>;
    using LD = Loads<XF4, WIN>;
    using SM = Smem<XF4, WIN>;
    static_assert(!HALF || XF4, "an MXFP8 step is 128 values");
    __shared__ __attribute__((aligned(16))) SM sm;
    __shared__ int s_prefix[kMaxGroups + 1];
    __shared__ int64_t s_offs[kMaxGroups + 1];   // no global load while the chain's are in flight
    __shared__ float s_rsw[SCALED ? 4 * 128 : 1];
    const int tid = threadIdx.x;
    const int lane_id = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int G = p.G;
    const int ntn = (int)((p.N + BN - 1) / BN);

    // tile table: prefix of the experts' tile counts (wave 0)
    if (wave == 0) {
        int cnt[kMaxGroups / 64];
        int local = 0;
#pragma unroll
        for (int u = 0; u < kMaxGroups / 64; ++u) {
            const int g = lane_id * (kMaxGroups / 64) + u;
            int c = 0;
            if (g < G) {
                const int64_t n = p.offs[g + 1] - p.offs[g];
                c = n > 0 ? (int)((n + BM - 1) / BM) * ntn : 0;
            }
            cnt[u] = c;
            local += c;
        }
        int incl = local;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(incl, d);
            if (lane_id >= d) incl += o;
        }
        int run = incl - local;
#pragma unroll
        for (int u = 0; u < kMaxGroups / 64; ++u) {
            const int g = lane_id * (kMaxGroups / 64) + u;
            if (g < G) {
                s_prefix[g] = run;
                run += cnt[u];
            }
        }
        if (lane_id == 63) s_prefix[G] = incl;
    }
    for (int g = tid; g <= G; g += NT4) s_offs[g] = p.offs[g];
    __syncthreads();
    const int total = uni(s_prefix[G]);
    // workgroup b runs on XCD b % 8: each XCD takes a contiguous run of tiles a round
    const int grid = gridDim.x, bid = blockIdx.x;
    const int slot = (grid % 8 == 0) ? (bid % 8) * (grid / 8) + bid / 8 : bid;

    // tiles walk bands of BAND M tiles, so that the tiles an XCD runs together
    // share x and w panels in its L2
    auto locate = [&](int t) -> Loc {
        int lo = 0, hi = G - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_prefix[mid] <= t) lo = mid; else hi = mid - 1;
        }
        const int g = lo, local = t - s_prefix[g];
        const int mtiles = (s_prefix[g + 1] - s_prefix[g]) / ntn;
        const int band = local / (BAND * ntn);
        const int rem = local - band * BAND * ntn;
        const int bm = min(BAND, mtiles - band * BAND);
        const int64_t m0 = s_offs[g] + (int64_t)(band * BAND + rem % bm) * BM;
        return Loc{uni(g), uni64(m0), uni64(min((int64_t)BM, s_offs[g + 1] - m0)), uni64((int64_t)(rem / bm) * BN)};
    };
    const int64_t lda = XF4 ? p.K / 2 : p.K, ldb = p.K / 2, lds = p.K / 32;
    const int nk_all = (int)((p.K + F::kBK - 1) / F::kBK);
    auto src_of = [&](const Loc& t) -> Src {
        const int64_t b0 = (int64_t)t.g * p.N + t.n0, nv = min((int64_t)BN, p.N - t.n0);
        return Src{make_rsrc(p.A.codes + t.m0 * lda, t.mvalid * lda), make_rsrc(p.B.codes + b0 * ldb, nv * ldb),
                   make_rsrc(p.A.scales + t.m0 * lds, t.mvalid * lds), make_rsrc(p.B.scales + b0 * lds, nv * lds),
                   nk_all};
    };

    if (slot < total) {
        const uint32_t smb = (uint32_t)uni((int)lds_addr(&sm));
        int w = slot;
        Loc L = locate(w);
        bool pre = false;
        int base = 0;          // stage of the tile's step 0
        int sbase = 0;         // and scale buffer of its window 0
        for (;;) {
            const int wnext = w + grid;
            const bool has_next = wnext < total;
            const int lane = lane_now();
            const int r16 = lane & 15, q = lane >> 4;
            const Src own = src_of(L);
            const int nk = nk_all;

            // ---- direct loads: a lane's offsets within a step ----
            // x, and w where a step has 128 bytes of a row: a load is 8 rows, lane
            // l fetches row l >> 3 and the chunk stored at l & 7.  w with 64-byte
            // steps: a load is 16 rows in 8 lines, lane l the 16 bytes stored at
            // chunk l & 7 of line l >> 3.
            const int lrow = lane >> 3, lchunk = (lane & 7) ^ lrow;
            const uint32_t aoff = (uint32_t)((wave * 64 + lrow) * lda + lchunk * 16);
            // MXFP4 x: rows 8..15 of each 16 (odd loads) have chunk lchunk ^ 1 there
            const uint32_t flip = (lchunk & 1) ? (uint32_t)-16 : 16u;
            const uint32_t boff =
                XF4 ? (uint32_t)((wave * 64 + lrow) * ldb + lchunk * 16)
                    : (uint32_t)((wave * 64 + lrow * 2 + (lchunk >> 2)) * ldb + (lchunk & 3) * 16);
            // scales: a window's 16 bytes of row wave * 64 + l; a step's kSub dwords:
            // lane l of load t fetches 4 bytes of row (t * 64 + l) / kSub
            const uint32_t soff = !WIN && XF4 ? (uint32_t)((wave * 64 + (lane >> 1)) * lds + (lane & 1) * 4)
                                              : (uint32_t)((wave * 64 + lane) * lds);
            const uint32_t over_c = HALF && lchunk >= 4 ? 0x80000000u : 0u;
            const uint32_t over_s = HALF && (lane & 1) ? 0x80000000u : 0u;
            // first scale byte of a step's window in its row: the last window ends
            // with the row
            auto win_byte = [&](int ks) {
                return min((uint32_t)(ks / F::kWin) * 16u, (uint32_t)lds - 16u);
            };
            // load u of step ks of a tile into stage st, scales into their buffer sb
            // (WIN: those of the window that starts at ks, if one does); LIVE: ks < nk is known
            auto dma = [&](auto uc, auto livec, const Src& s, int st, int sb, int ks) {
                constexpr int u = decltype(uc)::value;
                const bool live = decltype(livec)::value || ks < s.nk;
                const bool last = HALF && ks + 1 == s.nk;
                const uint32_t oc = HALF && last ? over_c : 0u, os = HALF && last ? over_s : 0u;
                auto rng = [&](const v4i& r) { return live ? r : v4i{r.x, r.y, 0, r.w}; };
                if constexpr (u < F::kALoads) {
                    dma_b128<u * 1024>(rng(s.ra), smb + (uint32_t)offsetof(SM, a) + st * (BM * 128) + wave * 8192,
                                       (aoff + (uint32_t)(u * 8 * lda) + (XF4 && (u & 1) ? flip : 0u)) | oc,
                                       (uint32_t)ks * 128u);
                } else if constexpr (u < F::kALoads + F::kBLoads) {
                    constexpr int v = u - F::kALoads;
                    dma_b128<v * 1024>(rng(s.rb),
                                       smb + (uint32_t)offsetof(SM, b) + st * (BN * F::kWBytes) +
                                           wave * (F::kBLoads * 1024),
                                       (boff + (uint32_t)(v * (XF4 ? 8 : 16) * ldb) + (XF4 && (v & 1) ? flip : 0u)) | oc,
                                       (uint32_t)ks * (uint32_t)F::kWBytes);
                } else {
                    constexpr int v = u - F::kCodeLoads;       // x scales, then w scales
                    constexpr bool isx = v < LD::kScale;
                    constexpr int t = isx ? v : v - LD::kScale;
                    const v4i r = rng(isx ? s.rsa : s.rsb);
                    const uint32_t at = smb + (uint32_t)(isx ? offsetof(SM, as) : offsetof(SM, bs));
                    if constexpr (WIN) {
                        // between window starts a load of no bytes, so that every step
                        // issues the same instructions
                        const bool start = ks % F::kWin == 0;
                        dma_b128(start ? r : v4i{r.x, r.y, 0, r.w},
                                 start ? at + sb * (BM * 16) + wave * 1024 : smb + (uint32_t)offsetof(SM, none),
                                 soff, win_byte(ks));
                    } else {
                        dma_b32<t * 256>(r, at + st * (BM * SM::kSRow) + wave * (256 * F::kSub),
                                         (soff + (uint32_t)(t * 32 * lds)) | os, (uint32_t)ks * (4u * F::kSub));
                    }
                }
            };

            // ---- fragments ----
            // lane (r16, q): row r16 of a block.  MXFP4 x: chunks 2q and 2q + 1 of
            // both operands, 32 values (one scale block) each, MFMA h of a block
            // taking chunk 2q + h of every lane and byte h of the lane's two scales.
            // MXFP8 x: x chunks q and q + 4 (K values 16q.. and 64 + 16q..), w chunk q
            // of its 64 bytes (values 32q..), scale byte q: the pairing of the mixed
            // MFMA.
            v4i af[8][2], bf[8][F::kSub];
            int asc[8], bsc[8];
            const int swz = (r16 & 7) ^ (XF4 ? r16 >> 3 : 0);
            const int a_row = wm * 128 + r16, b_row = wn * 128 + r16;
            const int ac0 = XF4 ? 2 * q : q, ac1 = XF4 ? 2 * q + 1 : q + 4;
            const int a0 = a_row * 128 + ((ac0 ^ swz) << 4), a1 = a_row * 128 + ((ac1 ^ swz) << 4);
            const int b0 = XF4 ? b_row * 128 + ((ac0 ^ swz) << 4)
                               : (b_row >> 1) * 128 + ((((r16 & 1) * 4 + q) ^ (r16 >> 1)) << 4);
            const int b1 = b_row * 128 + ((ac1 ^ swz) << 4);
            // those chunks' scales among the row's kept ones, from the step's first
            const int a_s = a_row * SM::kSRow + ac0, b_s = b_row * SM::kSRow + ac0;
            auto scales = [](const uint8_t* s) -> int {
                if constexpr (XF4) return *reinterpret_cast<const uint16_t*>(s);
                else return *s;
            };
            // where a step's fragments lie: its stage, and the offset of its scales
            struct Place {
                int st, s;
            };
            auto place = [&](int ks) -> Place {
                const int st = (base + ks) & 1;
                if constexpr (WIN)
                    return Place{st, ((sbase + ks / F::kWin) & 1) * (BM * SM::kSRow) +
                                         (int)((uint32_t)ks * (4u * F::kSub) - win_byte(ks))};
                else
                    return Place{st, st * (BM * SM::kSRow)};
            };
            auto read_a = [&](auto ic, const Place& p) {
                constexpr int i = decltype(ic)::value;
                af[i][0] = *reinterpret_cast<const v4i*>(sm.a[p.st] + a0 + i * 2048);
                af[i][1] = *reinterpret_cast<const v4i*>(sm.a[p.st] + a1 + i * 2048);
                asc[i] = scales(sm.as[0] + p.s + a_s + i * 16 * SM::kSRow);
            };
            auto read_b = [&](auto jc, const Place& p) {
                constexpr int j = decltype(jc)::value;
                bf[j][0] = *reinterpret_cast<const v4i*>(sm.b[p.st] + b0 + j * 16 * F::kWBytes);
                bsc[j] = scales(sm.bs[0] + p.s + b_s + j * 16 * SM::kSRow);
                if constexpr (XF4) bf[j][1] = *reinterpret_cast<const v4i*>(sm.b[p.st] + b1 + j * 2048);
            };
            // (WIN, HALF) the scale bytes read for chunks past K are some other
            // row's: zero them before the last step's MFMAs
            auto cut_scales = [&](int keep) {          // 0 or ~0
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    asc[i] &= keep;
                    bsc[i] &= keep;
                }
            };
            v4f acc[8][8];
            auto wide = [](const v4i& x) { return v8i{x.x, x.y, x.z, x.w, 0, 0, 0, 0}; };
            // Slot t of a pass over rows i0 .. i0 + 3: column t / 4.  MXFP8 x: row
            // t % 4.  MXFP4 x: two MFMAs, of rows 0 and 1 in slots 0 (first half of
            // their 256 values) and 1 (second half), rows 2 and 3 in slots 2 and 3:
            // the halves of a block follow each other at a distance of two, since
            // an MFMA whose input is the previous one's output would wait for it.
            // FIRST: the accumulation starts from zero.
            auto mfma = [&](auto tc, auto i0c, auto firstc) {
                constexpr int t = decltype(tc)::value, j = t / 4, i0 = decltype(i0c)::value;
                if constexpr (XF4) {
                    constexpr int h = t & 1, i = i0 + (t & 2);
                    static_for<2>([&](auto dc) {
                        constexpr int r = i + decltype(dc)::value;
                        const v4f c = decltype(firstc)::value && h == 0 ? v4f{0.f, 0.f, 0.f, 0.f} : acc[r][j];
                        acc[r][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            wide(bf[j][h * (F::kSub - 1)]), wide(af[r][h]), c, 4, 4, h, bsc[j], h, asc[r]);
                    });
                } else {
                    constexpr int i = i0 + t % 4;
                    const v8i x{af[i][0].x, af[i][0].y, af[i][0].z, af[i][0].w,
                                af[i][1].x, af[i][1].y, af[i][1].z, af[i][1].w};
                    const v4f c = decltype(firstc)::value ? v4f{0.f, 0.f, 0.f, 0.f} : acc[i][j];
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(bf[j][0]), x, c, 4, 0, 0,
                                                                                 bsc[j], 0, asc[i]);
                }
            };
            // The accumulators take all 256 AGPRs.  Held there between the steps,
            // each MXFP4 block keeps its registers through its two MFMAs; left to
            // itself the compiler gave the first one's result others and moved some
            // 130 registers a step.
            auto pin = [&]() {
                if constexpr (XF4) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int j = 0; j < 8; ++j) asm volatile("" : "+a"(acc[i][j]));
                }
            };
            // K step ks with the loads of step kl of s into the stage it frees.
            // First pass: rows 0..3, the stage is free after the barrier (every
            // wave holds its fragments).  Then this wave's loads of step ks + 1 have
            // landed (only the first pass's newer ones may be in flight), and after
            // the barrier everybody's: the second pass (rows 4..7) reads the next
            // fragments into the registers its MFMAs free.
            // sb: the scale buffer for the window that starts at step kl of s.
            auto step = [&](int ks, auto livec, const Src& s, int sb, int kl, auto firstc) {
                const int cur = (base + ks) & 1;
                lds_barrier();
                if constexpr (WIN && HALF) cut_scales(ks + 1 == nk && q >= 2 ? 0 : ~0);
                static_for<32>([&](auto sc) {
                    constexpr int t = decltype(sc)::value;
                    mfma(sc, std::integral_constant<int, 0>{}, firstc);
                    __builtin_amdgcn_sched_barrier(0);
                    constexpr int u = load_at_a<XF4>(t);
                    if constexpr (u >= 0) dma(std::integral_constant<int, u>{}, livec, s, cur, sb, kl);
                    __builtin_amdgcn_sched_barrier(0);
                });
                wait_vm<F::kNA>();
                lds_barrier();
                const Place nxt = place(ks + 1);
                static_for<32>([&](auto sc) {
                    constexpr int t = decltype(sc)::value, j = t / 4;
                    mfma(sc, std::integral_constant<int, 4>{}, firstc);
                    __builtin_amdgcn_sched_barrier(0);
                    if constexpr (t < 4) read_a(std::integral_constant<int, t>{}, nxt);
                    // in the last column a row is read once its last MFMA has issued
                    if constexpr (t >= 28 && !XF4) read_a(std::integral_constant<int, 4 + t % 4>{}, nxt);
                    if constexpr (t >= 28 && XF4 && t % 2 == 1) {
                        read_a(std::integral_constant<int, 4 + (t & 2)>{}, nxt);
                        read_a(std::integral_constant<int, 5 + (t & 2)>{}, nxt);
                    }
                    if constexpr (t % 4 == 3) read_b(std::integral_constant<int, j>{}, nxt);
                    constexpr int u = load_at_b<XF4, WIN>(t);
                    if constexpr (u >= 0) dma(std::integral_constant<int, u>{}, livec, s, cur, sb, kl);
                    __builtin_amdgcn_sched_barrier(0);
                });
            };

            if (!pre) {
                wait_vm<0>();
                lds_barrier();                     // no load in flight, stages free
            }
            if constexpr (SCALED) {
                // the wave's 128 row scales (rows past the tile read 0); the previous
                // tile's epilogue has read its own, and the first step's wait covers
                // these loads
                const int64_t n = min((int64_t)128, max((int64_t)0, L.mvalid - wm * 128));
                const v4i rr = make_rsrc(p.rscale + L.m0 + wm * 128, n * 4);
                const uint32_t la = (uint32_t)uni((int)lds_addr(&s_rsw[wave * 128]));
                dma_b32(rr, la, (uint32_t)lane * 4u, 0u);
                dma_b32(rr, la + 256u, (uint32_t)lane * 4u + 256u, 0u);
            }
            if (!pre) {
                static_for<LD::kAll>([&](auto uc) { dma(uc, std::false_type{}, own, base, sbase, 0); });
                static_for<LD::kAll>([&](auto uc) { dma(uc, std::false_type{}, own, base ^ 1, sbase, 1); });
                wait_vm<LD::kAll>();
                lds_barrier();
            }
            const Place first = place(0);
            static_for<8>([&](auto ic) { read_a(ic, first); });
            static_for<8>([&](auto jc) { read_b(jc, first); });
            auto buf = [&](int ks) { return WIN ? (sbase + ks / F::kWin) & 1 : 0; };
            const int snext = WIN ? (sbase + (nk + F::kWin - 1) / F::kWin) & 1 : 0;   // the next tile's
            int ks = 0;
            if (nk >= 3) {
                step(0, std::true_type{}, own, buf(2), 2, std::true_type{});
                ks = 1;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
            }
            for (; ks + 2 < nk; ++ks) {
                pin();
                step(ks, std::true_type{}, own, buf(ks + 2), ks + 2, std::false_type{});
                pin();
            }
            Loc Ln = L;
            Src nx = own;
            nx.nk = 0;                             // no next tile: zero-range loads
            if (has_next) {
                Ln = locate(wnext);
                nx = src_of(Ln);
            }
            for (; ks < nk; ++ks) {
                pin();
                step(ks, std::false_type{}, nx, snext, ks + 2 - nk, std::false_type{});
                pin();
            }
            store_tile_bf16_regs<SCALED>(acc, p, L.g, L.m0, L.mvalid, L.n0, wm, wn, lane_now(), 1.0f,
                                         SCALED ? &s_rsw[wave * 128] : nullptr);
            if (!has_next) break;
            pre = nk >= 2;                         // a one-step tile loads nothing ahead
            base = uni(pre ? (base + nk) & 1 : 0);
            sbase = uni(pre ? snext : 0);
            w = wnext;
            L = Ln;
        }
    }
    // no load may still be landing in LDS when the workgroup ends
    wait_vm<0>();
}

template <bool XF4, bool HALF, bool WIN>
void launch_tile(const GemmProblem& p, int grid, hipStream_t s) {
    if (p.rscale)
        hipLaunchKernelGGL((linear4_tile_kernel<XF4, HALF, WIN, true>), dim3(grid), dim3(NT4), 0, s, p);
    else
        hipLaunchKernelGGL((linear4_tile_kernel<XF4, HALF, WIN, false>), dim3(grid), dim3(NT4), 0, s, p);
}

}  // namespace

hipError_t launch_linear4_tile(bool x_fp4, const GemmProblem& p, hipStream_t s) {
    int grid = device_cu_count();
    grid = grid < 8 ? 8 : grid / 8 * 8;
    const bool win = p.K >= 512, half = p.K % 256 != 0;
    if (!x_fp4) win ? launch_tile<false, false, true>(p, grid, s) : launch_tile<false, false, false>(p, grid, s);
    else if (half) win ? launch_tile<true, true, true>(p, grid, s) : launch_tile<true, true, false>(p, grid, s);
    else win ? launch_tile<true, false, true>(p, grid, s) : launch_tile<true, false, false>(p, grid, s);
    return hipGetLastError();
}

}  // namespace mx
