// GroupedLinear on MXFP4 weights for few rows an expert, and the whole MoE
// layer for a few tokens (gfx950).  Both stream the weights once through the
// core in few_rows.h.
//
// The layer runs as three or four launches on one stream:
//  * layer_prep: workgroup 0 routes (top-k by a bitwise search for the k-th
//    largest key, softmax of the selected logits) and lists the routed rows
//    sorted by (expert, token); the other workgroups quantize one token of x
//    each to MXFP8 (MX weights only).
//  * layer_gate_up: a workgroup takes 32 columns of F of one routed expert (64
//    rows of W1), its four waves a quarter of H each; z = r silu(a) b leaves
//    as MXFP8 blocks (MX weights) or bf16.
//  * layer_down: a workgroup takes 16, 32 or 64 rows of every routed expert's
//    W2, or a share of their products where few such rows would leave CUs idle,
//    and adds the experts' products in fp32 in LDS: the combine needs no atomics
//    and has one fixed order.
//  * layer_sum: adds those shares, where there are any.
// Sums are fp32 of exact products in all formats.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "few_rows.h"
#include "gemm_device.h"
#include "internal.h"
#include "mx_device.h"

namespace mx {
namespace {

using namespace few;

// ---- GroupedLinear, few rows an expert --------------------------------------

constexpr int kLinRows = 64;      // rows of W (columns of y) per unit
constexpr int kLinWaves = 4;

struct LinearArgs {
    const uint8_t *x, *xs, *w, *ws;
    const int64_t* offs;
    const float* rscale;
    uint16_t* y;
    int64_t N, K;
    int G;
};

// A workgroup's units: 64 columns of y for up to 16 NT rows of one expert, the
// four waves a quarter of K each.  Units run over (expert with rows, column
// block), and over an expert's row chunks within one: rows that an expert has
// beyond a chunk lengthen its workgroups' turn instead of filling other CUs.
// Made for few rows, where the weights' one reading is the time (16 rows on 8 x
// (28672, 4096): 78 us, 5.6 TB/s); 16384 rows of K = 2880 on one expert of 4096
// columns (64 workgroups, 256 turns) take 2.2 ms, as 256 x 256 tiles of K = 2944
// 0.12.
template <int XF, int NT, int kSteps, bool FULL, bool ODD>
__global__ void __launch_bounds__(64 * kLinWaves, 2)
linear4_few_kernel(LinearArgs p) {
    __shared__ __attribute__((aligned(16))) float parts[2][kLinWaves * 1024];
    __shared__ int s_count;
    __shared__ int64_t s_lo[kMaxGroups], s_hi[kMaxGroups];    // experts with rows, in order
    __shared__ int s_e[kMaxGroups];
    const int tid = threadIdx.x, wave = uni(tid >> 6), lane = tid & 63;
    if (wave == 0) {
        int n = 0;
        for (int e0 = 0; e0 < p.G; e0 += 64) {
            const int e = e0 + lane;
            int64_t lo = 0, hi = 0;
            if (e < p.G) {
                lo = p.offs[e];
                hi = p.offs[e + 1];
            }
            const uint64_t has = __ballot(hi > lo);
            if (hi > lo) {
                const int at = n + __popcll(has & ((1ull << lane) - 1));
                s_e[at] = e;
                s_lo[at] = lo;
                s_hi[at] = hi;
            }
            n += __popcll(has);
        }
        if (lane == 0) s_count = n;
    }
    __syncthreads();
    const int ncol = (int)((p.N + kLinRows - 1) / kLinRows);
    const int64_t units = (int64_t)uni(s_count) * ncol;
    const int steps = (int)((p.K + 127) / 128);
    // waves past the number of groups repeat the first one; their sums are not added
    const int waves = min(kLinWaves, FULL ? steps / kSteps : steps);
    int s0, s1;
    share<kSteps, FULL>(steps, wave < waves ? wave : 0, waves, s0, s1);
    using U = Unit<4>;
    auto place = [&](U& u, int id, int64_t m0) -> bool {      // rows from m0, or the expert's first (m0 < 0)
        if (id >= units) return false;
        const int i = id / ncol;
        const int64_t n0 = (int64_t)(id - i * ncol) * kLinRows;
        const int64_t e = uni(s_e[i]);
        const int64_t lo = uni64(s_lo[i]), hi = uni64(s_hi[i]);
        u.row0 = m0 < 0 ? lo : m0;
        u.rows = (int)min((int64_t)(16 * NT), hi - u.row0);
        u.s0 = s0;
        u.s1 = s1;
        u.id = id;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            // tiles past N (N % 32 == 0) repeat the first one and are not stored
            const int64_t r = e * p.N + (n0 + 16 * t < p.N ? n0 + 16 * t : n0);
            u.wc[t] = p.w + r * (p.K / 2);
            u.ws[t] = p.ws + r * (p.K / 32);
        }
        return true;
    };
    int turn = 0;
    float scale[NT];                 // row scale of this thread's token in done
    stream<kFp4, XF, 4, NT, kSteps, FULL, ODD, false>(
        p.K, lane, [&](U& u) { return place(u, blockIdx.x, -1); },
        [&](U& u) {
            const int64_t hi = uni64(s_hi[u.id / ncol]);
            if (u.row0 + 16 * NT < hi) return place(u, u.id, u.row0 + 16 * NT);
            return place(u, u.id + (int)gridDim.x, -1);
        },
        [&](const U& u, int n) {
            return x_row<XF>(p.x, p.xs, u.row0 + min(n * 16 + (lane & 15), u.rows - 1), p.K, lane);
        },
        [&](const U& u) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
                scale[n] = p.rscale ? p.rscale[u.row0 + min(n * 16 + (tid >> 4), u.rows - 1)] : 1.0f;
        },
        [&](const v4f(&acc)[4][NT], const U& u) {
            const int64_t n0 = (int64_t)(u.id % ncol) * kLinRows;
            // the waves' K parts, added in wave order; thread (token, 4 columns).  Two
            // buffers in turn: a wave that writes one has passed the barrier of the
            // other, and with it everybody's reads of this one.
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n * 16 >= u.rows) break;
                float* const part = parts[turn];
                turn ^= 1;
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    *reinterpret_cast<v4f*>(part + ((wave * 4 + t) * 64 + lane) * 4) = acc[t][n];
                lds_barrier();       // (__syncthreads would wait for the weights in flight)
                const int tok = tid >> 4, c4 = tid & 15;          // columns n0 + 4 c4 .. + 3
                const int at = ((c4 >> 2) * 64 + (c4 & 3) * 16 + tok) * 4;
                v4f s = *reinterpret_cast<const v4f*>(part + at);
#pragma unroll
                for (int v = 1; v < kLinWaves; ++v)
                    if (v < waves) s += *reinterpret_cast<const v4f*>(part + v * 1024 + at);
                const int row = n * 16 + tok;
                const int64_t col = n0 + 4 * c4;
                if (row < u.rows && col < p.N) {
                    const float f = scale[n];
                    *reinterpret_cast<uint2*>(p.y + (u.row0 + row) * p.N + col) =
                        make_uint2(bf16x2(s[0] * f, s[1] * f), bf16x2(s[2] * f, s[3] * f));
                }
            }
        });
}

// ---- the layer: plan ---------------------------------------------------------

constexpr int kPrepThreads = 1024;

// order-preserving key of a logit: larger float, larger key; equal floats (0
// and -0 among them), equal keys; NaN and -inf 0
__device__ __forceinline__ uint32_t logit_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);       // -0 + 0 is 0
    if (!(v > -__builtin_inff())) return 0u;
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// Reductions over a wave's 64 lanes, every lane with the result: DPP within rows
// of 16, then swaps 16 and 32 lanes apart (no LDS traffic, unlike a shuffle).
template <class Op>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, Op op) {
    v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));     // lanes ^ 1
    v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));     // lanes ^ 2
    v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x124, 0xF, 0xF, false));    // row_ror:4
    v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x128, 0xF, 0xF, false));    // row_ror:8
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return op(b[0], b[1]);
}

// Workgroup 0 of layer_prep.  LDS: the selected experts of each token as bits,
// each expert's rows, and each token's routing weights.  W: 64-expert words per
// token that the registers hold (1 for E <= 64, else the largest).
template <int W>
__device__ void layer_plan(const float* __restrict__ logits, int T, int E, int k, const LayerPlan& plan,
                           uint8_t* smem) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int words = (E + 63) / 64;                                     // 64-expert words per token
    uint64_t* sel = reinterpret_cast<uint64_t*>(smem);                   // [T][words]
    int* cnt = reinterpret_cast<int*>(sel + (int64_t)T * words);         // [E] rows, then first rows
    float* wt = reinterpret_cast<float*>(cnt + E);                       // [T][k] weights, by expert
    auto read = [&](float (&v)[W], int t) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int e = lane + 64 * i;
            v[i] = t < T && e < E ? logits[(int64_t)t * E + e] : -__builtin_inff();
        }
    };
    float ahead[W];                      // the next token's logits
    read(ahead, wave);
    for (int t = wave; t < T; t += kPrepThreads / 64) {
        uint32_t key[W];
#pragma unroll
        for (int i = 0; i < W; ++i) key[i] = logit_key(ahead[i]);
        read(ahead, t + kPrepThreads / 64);
        // th: the largest value that at least k keys reach (0 if fewer routed), or,
        // as soon as a value splits off exactly k keys, the one below it
        uint32_t th = 0;
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t cand = th | (1u << bit);
            int n = 0;
#pragma unroll
            for (int i = 0; i < W; ++i) n += __popcll(__ballot(key[i] >= cand));
            if (n == k) {
                th = cand - 1;
                break;
            }
            if (n > k) th = cand;
        }
        int above = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) above += __popcll(__ballot(key[i] > th));
        // keys above th, and of those equal to it the first k - above by index
        // (th == 0: the rest are masked experts, and none of them is taken)
        int left = th ? k - above : 0;
        uint32_t top = 0;
        uint64_t mine = 0;
        bool on[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint64_t eq = __ballot(key[i] == th);
            on[i] = key[i] > th || (key[i] == th && __popcll(eq & ((1ull << lane) - 1)) < left);
            left -= min(left, (int)__popcll(eq));
            const uint64_t b = __ballot(on[i]);
            if (lane == i) mine = b;
            if (on[i]) top = max(top, key[i]);
        }
        top = wave_reduce(top, [](uint32_t a, uint32_t b) { return max(a, b); });
        const float m = key_logit(top);
        float ex[W], sum = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            ex[i] = on[i] ? expf(key_logit(key[i]) - m) : 0.f;
            sum += ex[i];
        }
        sum = __uint_as_float(wave_reduce(__float_as_uint(sum), [](uint32_t a, uint32_t b) {
            return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
        }));
        if (lane < words) sel[t * words + lane] = mine;
        int before = 0;                  // selected experts below this lane's
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint64_t b = __ballot(on[i]);
            if (on[i]) wt[t * k + before + __popcll(b & ((1ull << lane) - 1))] = ex[i] / sum;
            before += __popcll(b);
        }
    }
    __syncthreads();
    // An expert's tokens: by one thread for each expert, token by token (about 40
    // cycles each), or by one of the 16 waves, 64 tokens in a ballot (about 150):
    // the first where 4 T < E for every 64 tokens.
    const bool by_thread = 4 * T < E * ((T + 63) / 64);
    auto routed = [&](int t, int e) { return (sel[t * words + (e >> 6)] >> (e & 63) & 1) != 0; };
    auto place = [&](int row, int t, int e) {
        plan.tok[row] = t;
        int slot = 0;
        for (int i = 0; i < (e >> 6); ++i) slot += __popcll(sel[t * words + i]);
        slot += __popcll(sel[t * words + (e >> 6)] & ((1ull << (e & 63)) - 1));
        plan.r[row] = wt[t * k + slot];
    };
    auto tokens = [&](int e, int t0) -> uint64_t {
        const int t = t0 + lane;
        return __ballot(t < T && routed(t, e));
    };
    if (by_thread) {
        for (int e = tid; e < E; e += kPrepThreads) {
            int n = 0;
            for (int t = 0; t < T; ++t) n += routed(t, e);
            cnt[e] = n;
        }
    } else for (int e = wave; e < E; e += kPrepThreads / 64) {
        int n = 0;
        for (int t0 = 0; t0 < T; t0 += 64) n += __popcll(tokens(e, t0));
        if (lane == 0) cnt[e] = n;
    }
    __syncthreads();
    // wave 0: first row of each expert and the list of routed experts
    if (wave == 0) {
        int rows = 0, act = 0;
        for (int i = 0; i < words; ++i) {
            const int e = lane + 64 * i;
            const int n = e < E ? cnt[e] : 0;
            int incl = n;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(incl, d);
                if (lane >= d) incl += o;
            }
            const uint64_t has = __ballot(n > 0);
            const int first = rows + incl - n;
            if (n > 0)
                plan.act[act + __popcll(has & ((1ull << lane) - 1))] = make_int4(e, first, n, 0);
            if (e < E) cnt[e] = first;
            rows += __shfl(incl, 63);
            act += __popcll(has);
        }
        if (lane == 0) *plan.n_act = act;
    }
    __syncthreads();
    // rows: an expert's tokens in order, with their routing weights
    if (by_thread) {
        for (int e = tid; e < E; e += kPrepThreads) {
            int row = cnt[e];
            for (int t = 0; t < T; ++t)
                if (routed(t, e)) place(row++, t, e);
        }
    } else for (int e = wave; e < E; e += kPrepThreads / 64) {
        int row = cnt[e];
        for (int t0 = 0; t0 < T; t0 += 64) {
            const uint64_t b = tokens(e, t0);
            const int t = t0 + lane;
            if (b >> lane & 1) place(row + __popcll(b & ((1ull << lane) - 1)), t, e);
            row += __popcll(b);
        }
    }
}

size_t prep_lds(int64_t T, int E, int k) {
    return (size_t)(T * ((E + 63) / 64) * 8 + E * 4 + T * k * 4);
}

// MXFP8 blocks of one token (H % 128 == 0), as mxfp8_quantize makes them; a
// block with an infinity or a NaN becomes NaNs, so that the token's output says
// so.
__device__ void quant_token(const uint16_t* __restrict__ x, int H, uint8_t* __restrict__ codes,
                            uint8_t* __restrict__ scales) {
    for (int u = threadIdx.x; u < H / 8; u += kPrepThreads) {
        const uint4 p = *reinterpret_cast<const uint4*>(x + u * 8);
        const uint32_t w[4] = {p.x, p.y, p.z, p.w};
        float v[8];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            m = max(m, max(abs_bits(v[2 * i]), abs_bits(v[2 * i + 1])));
        }
        m = max(m, (uint32_t)__shfl_xor((int)m, 1));       // a block is four lanes
        m = max(m, (uint32_t)__shfl_xor((int)m, 2));
        const bool bad = m >= 0x7f800000u;
        const uint32_t c = scale_code_from_amax_bits(m);
        const float lim = e4m3_limit_from_code(c), s = scale_from_code(c);
        uint2 o = make_uint2(e4m3x4_scaled(v[0], v[1], v[2], v[3], lim, s),
                             e4m3x4_scaled(v[4], v[5], v[6], v[7], lim, s));
        if (bad) o = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
        *reinterpret_cast<uint2*>(codes + u * 8) = o;
        if ((threadIdx.x & 3) == 0) scales[u >> 2] = bad ? 127 : (uint8_t)c;
    }
}

__global__ void __launch_bounds__(kPrepThreads)
layer_prep_kernel(LayerArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    if (blockIdx.x == 0) {
        if (p.E <= 64) layer_plan<1>(p.logits, (int)p.T, p.E, p.k, p.plan, smem);
        else layer_plan<kMaxGroups / 64>(p.logits, (int)p.T, p.E, p.k, p.plan, smem);
    } else {
        const int64_t t = blockIdx.x - 1;
        quant_token(p.x + t * p.H, (int)p.H, p.xq + t * p.H, p.xqs + t * (p.H / 32));
    }
}

// ---- the layer: gate-up --------------------------------------------------------

constexpr int kGuWaves = 4;

// LDS copy of the plan: the routed experts and the rows' tokens.
struct PlanLds {
    int4* act;
    int* tok;
    float* r;
    int n_act;
};
size_t plan_lds_bytes(const LayerArgs& p) {
    const int64_t rows = p.T * p.k, experts = p.E < rows ? p.E : rows;
    return (size_t)(experts * 16 + rows * 8);
}
__device__ __forceinline__ PlanLds read_plan(const LayerArgs& p, uint8_t* smem) {
    const int rows = (int)p.T * p.k, experts = min(p.E, rows);
    PlanLds l{reinterpret_cast<int4*>(smem), reinterpret_cast<int*>(smem + experts * 16),
              reinterpret_cast<float*>(smem + experts * 16 + rows * 4), 0};
    // (entries past the routed ones are not initialised and not used)
    for (int i = threadIdx.x; i < experts; i += blockDim.x) l.act[i] = p.plan.act[i];
    for (int i = threadIdx.x; i < rows; i += blockDim.x) {
        l.tok[i] = p.plan.tok[i];
        l.r[i] = p.plan.r[i];
    }
    l.n_act = uni(*p.plan.n_act);
    __syncthreads();
    return l;
}

// A workgroup's units: 32 columns of z (tiles 0, 1: their gate rows of W1; 2, 3:
// the up rows) for up to 16 NT rows of one routed expert, the four waves a
// quarter of H each.
template <int WF, int NT, int kSteps, bool FULL>
__global__ void __launch_bounds__(64 * kGuWaves, 2)
layer_gate_up_kernel(LayerArgs p) {
    constexpr int XF = WF == kBf16 ? kBf16 : kFp8;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    __shared__ __attribute__((aligned(16))) float parts[2][kGuWaves * 1024];
    const int tid = threadIdx.x, wave = uni(tid >> 6), lane = tid & 63;
    const PlanLds plan = read_plan(p, smem);
    const int ncol = (int)(p.F / 32), units = plan.n_act * ncol;
    const int steps = (int)(p.H / 128);
    // waves past the number of groups repeat the first one; their sums are not added
    const int waves = min(kGuWaves, FULL ? steps / kSteps : steps);
    int s0, s1;
    share<kSteps, FULL>(steps, wave < waves ? wave : 0, waves, s0, s1);
    const int64_t wb = row_bytes(WF, p.H), sb = p.H / 32;
    using U = Unit<4>;
    auto place = [&](U& u, int id, int c0) -> bool {       // the expert's rows from its c0-th
        if (id >= units) return false;
        const int a = id / ncol;
        const int4 ex = plan.act[a];
        const int64_t e = uni(ex.x);
        u.row0 = uni(ex.y) + c0;
        u.rows = min(16 * NT, uni(ex.z) - c0);
        u.s0 = s0;
        u.s1 = s1;
        u.id = id;
        const int64_t f0 = (int64_t)(id - a * ncol) * 32;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int64_t r = e * 2 * p.F + (t >> 1) * p.F + f0 + (t & 1) * 16;
            u.wc[t] = p.w1 + r * wb;
            u.ws[t] = WF == kBf16 ? nullptr : p.w1s + r * sb;
        }
        return true;
    };
    int turn = 0;
    stream<WF, XF, 4, NT, kSteps, FULL, false, WF != kBf16>(
        p.H, lane, [&](U& u) { return place(u, blockIdx.x, 0); },
        [&](U& u) {
            const int4 ex = plan.act[u.id / ncol];
            const int c0 = (int)u.row0 - uni(ex.y) + 16 * NT;
            if (c0 < uni(ex.z)) return place(u, u.id, c0);
            return place(u, u.id + (int)gridDim.x, 0);
        },
        [&](const U& u, int n) {
            const int tok = plan.tok[(int)u.row0 + min(n * 16 + (lane & 15), u.rows - 1)];
            if constexpr (WF == kFp4) return x_row_run(p.xq, p.xqs, tok, p.H, lane);
            else
                return x_row<XF>(WF == kBf16 ? reinterpret_cast<const uint8_t*>(p.x) : p.xq, p.xqs, tok, p.H,
                                 lane);
        },
        [](const U&) {},
        [&](const v4f(&acc)[4][NT], const U& u) {
            const int64_t f0 = (int64_t)(u.id % ncol) * 32;
            // a thread's places, computed here: kept through the stream they would
            // take registers that it has not got
            int me = tid;
            asm volatile("" : "+v"(me));
            // (buffers in turn as in linear4_few_kernel)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n * 16 >= u.rows) break;
                float* const part = parts[turn];
                turn ^= 1;
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    *reinterpret_cast<v4f*>(part + ((wave * 4 + t) * 64 + lane) * 4) = acc[t][n];
                // thread (token, two columns f0 + 2 c, + 1): the 16 threads of a token
                // are one DPP row and hold one block of 32
                const int tok = me >> 4, c = (me & 15) * 2;
                const int row = n * 16 + tok;
                const bool live = row < u.rows;
                const int64_t zrow = u.row0 + row;
                const float r = live ? plan.r[zrow] : 0.f;
                lds_barrier();
                const int at = ((c >> 4) * 64 + ((c & 15) >> 2) * 16 + tok) * 4 + (c & 3);
                float g[2] = {0.f, 0.f}, up[2] = {0.f, 0.f};
#pragma unroll
                for (int v = 0; v < kGuWaves; ++v)
                    if (v < waves) {
                        const float2 a = *reinterpret_cast<const float2*>(part + v * 1024 + at);
                        const float2 b = *reinterpret_cast<const float2*>(part + v * 1024 + 512 + at);
                        g[0] += a.x;
                        g[1] += a.y;
                        up[0] += b.x;
                        up[1] += b.y;
                    }
                // (the hardware's exp and reciprocal, as in the GroupedMLP's epilogue:
                // silu is off by at most some (|g| + 4) 2^-23 of itself, 1e-6 for
                // usual g, against the 2^-4 (bf16: 2^-8) of z's own rounding)
                float z[2];
#pragma unroll
                for (int v = 0; v < 2; ++v)
                    z[v] = r * (g[v] * __builtin_amdgcn_rcpf(1.0f + __expf(-g[v])) * up[v]);
                if constexpr (WF == kBf16) {
                    if (live)
                        *reinterpret_cast<uint32_t*>(p.z + (zrow * p.F + f0 + c) * 2) = bf16x2(z[0], z[1]);
                } else {
                    uint32_t m = max(abs_bits(z[0]), abs_bits(z[1]));
                    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, false));
                    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, false));
                    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x124, 0xF, 0xF, false));
                    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x128, 0xF, 0xF, false));
                    const bool bad = m >= 0x7f800000u;
                    const uint32_t sc = bad ? 127u : scale_code_from_amax_bits(m);
                    const uint32_t o = bad ? 0x7f7fu : e4m3x2_scaled(0u, z[0], z[1], e4m3_limit_from_code(sc),
                                                                     scale_from_code(sc), false);
                    if (live) {
                        *reinterpret_cast<uint16_t*>(p.z + zrow * p.F + f0 + c) = (uint16_t)o;
                        if (c == 0) p.zs[zrow * (p.F / 32) + f0 / 32] = (uint8_t)sc;
                    }
                }
            }
        });
}

// ---- the layer: down and combine -------------------------------------------------

constexpr int kDnWaves = 8;
// Workgroups of the down projection: one a CU.  64 tokens on 64 x (2048, 1408) MXFP4,
// 128 / 256 / 384 / 512 workgroups: 43 / 28 / 46 / 38 us (a workgroup's eight waves
// take a CU's registers, so more of them run one after the other).
constexpr int kSplitFull = 256;

// LDS of a down-projection workgroup: the plan, and its waves' sums of T tokens
// by 16 rt columns.
size_t down_lds(int64_t T, int k, int E, int rt) {
    const int64_t rows = T * k, experts = E < rows ? E : rows;
    return (size_t)(experts * 16 + rows * 8 + (int64_t)kDnWaves * T * 16 * rt * 4);
}
constexpr size_t kLdsBytes = 160 * 1024;

// 16-row tiles of W2 a workgroup takes; z is read once for all of them, and for
// MX weights one tile of z rows is as many bytes (MXFP4: twice) as one tile of
// W2.  One tile: H / 16 workgroups fill the CUs and no sums of parts are left to
// add.  Whole layer in us, one / two / four tiles: 8 x (4096, 14336), top 2, MXFP4
// 1 token 52 / 54 / 54, 4 102 / 103 / 103, 16 155 / 151 / 153, 32 178 / 166 / 164,
// 33 191 / 180 / 182, 64 236 / 210 / 207; MXFP8 4 155 / 157 / 157, 16 275 / 269 /
// 267, 32 294 / 282 / 279, 33 321 / 309 / 322, 64 369 / 346 / 355; 64 x (2048,
// 1408), top 8, MXFP4 1 25 / 25 / 30, 16 77 / 79 / 75, 32 82 / 79 / 84, 64 89 / 85 /
// 90; MXFP8 1 28 / 29 / 32, 64 130 / 126 / 126.  bf16, 16 tokens, all experts of 8 x
// (4096, 14336), the down projection alone: 155 / 156 / 170.
int down_tiles(bool bf16, int64_t T, int k, int E) {
    int rt = T <= 4 || (bf16 && T <= 16) ? 1 : T <= 16 || T > 32 || bf16 ? 2 : 4;
    while (rt > 1 && down_lds(T, k, E, rt) > kLdsBytes) rt /= 2;
    return rt;
}

// `split` workgroups share rows h0 .. h0 + 16 RT - 1 of every routed expert's W2.  Their
// waves' units are (expert, part of F, chunk of rows); each wave adds its units'
// products to its own sums[token][16 RT], and the waves' sums are added in order.
// With split > 1 a workgroup leaves its sums in `parts` and layer_sum adds them.
// (Adding them in the last workgroup to arrive took six times as long: the
// fences that such a hand-over needs write the XCD's L2 back, 0.3 us each.)
template <int WF, int NT, int kSteps, bool FULL, int RT>
__global__ void __launch_bounds__(64 * kDnWaves, 2)
layer_down_kernel(LayerArgs p) {
    constexpr int XF = WF == kBf16 ? kBf16 : kFp8;
    constexpr int kCols = 16 * RT;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, wave = uni(tid >> 6), lane = tid & 63;
    const int64_t h0 = (int64_t)(blockIdx.x / p.split) * kCols;
    const int part = blockIdx.x % p.split, waves = kDnWaves * p.split;
    const int T = (int)p.T;
    float* const sums = reinterpret_cast<float*>(smem);        // [wave][T][kCols]
    float* const out = sums + wave * T * kCols;
    for (int i = lane; i < T * 4 * RT; i += 64) reinterpret_cast<v4f*>(out)[i] = v4f{0.f, 0.f, 0.f, 0.f};
    const PlanLds plan = read_plan(p, smem + kDnWaves * T * kCols * 4);
    const int steps = (int)(p.F / 128);
    // parts of F per expert, so that every wave has work with few experts
    const int parts = max(1, min(FULL ? steps / kSteps : (steps + kSteps - 1) / kSteps,
                                 (2 * waves + plan.n_act - 1) / max(plan.n_act, 1)));
    const int units = plan.n_act * parts;
    const int64_t wb = row_bytes(WF, p.F), sb = p.F / 32;
    using U = Unit<RT>;
    auto place = [&](U& u, int id, int c0) -> bool {
        if (id >= units) return false;
        const int a = id / parts, c = id - a * parts;
        const int4 ex = plan.act[a];
        u.row0 = uni(ex.y) + c0;
        u.rows = min(16 * NT, uni(ex.z) - c0);
        share<kSteps, FULL>(steps, c, parts, u.s0, u.s1);
        u.id = id;
        const int64_t r = (int64_t)uni(ex.x) * p.H + h0;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            u.wc[t] = p.w2 + (r + 16 * t) * wb;
            u.ws[t] = WF == kBf16 ? nullptr : p.w2s + (r + 16 * t) * sb;
        }
        return true;
    };
    stream<WF, XF, RT, NT, kSteps, FULL, false, WF != kBf16>(
        p.F, lane, [&](U& u) { return place(u, part * kDnWaves + wave, 0); },
        [&](U& u) {
            const int4 ex = plan.act[u.id / parts];
            const int c0 = (int)u.row0 - uni(ex.y) + 16 * NT;
            if (c0 < uni(ex.z)) return place(u, u.id, c0);
            return place(u, u.id + waves, 0);
        },
        [&](const U& u, int n) {
            const int64_t row = u.row0 + min(n * 16 + (lane & 15), u.rows - 1);
            if constexpr (WF == kFp4) return x_row_run(p.z, p.zs, row, p.F, lane);
            else return x_row<XF>(p.z, p.zs, row, p.F, lane);
        },
        [](const U&) {},
        [&](const v4f(&acc)[RT][NT], const U& u) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int row = n * 16 + (lane & 15);
                if (row < u.rows) {       // an expert's tokens are distinct: no two lanes share a sum
                    float* o = out + plan.tok[(int)u.row0 + row] * kCols + 4 * (lane >> 4);
#pragma unroll
                    for (int t = 0; t < RT; ++t) *reinterpret_cast<v4f*>(o + 16 * t) += acc[t][n];
                }
            }
        });
    __syncthreads();
    for (int i = tid; i < T * 8 * RT; i += 64 * kDnWaves) {        // two columns of a token a thread
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < kDnWaves; ++v) {
            const float2 a = *reinterpret_cast<const float2*>(sums + v * T * kCols + 2 * i);
            s.x += a.x;
            s.y += a.y;
        }
        const int64_t at = (int64_t)(i / (8 * RT)) * p.H + h0 + 2 * (i % (8 * RT));
        if (p.split == 1) *reinterpret_cast<uint32_t*>(p.out + at) = bf16x2(s.x, s.y);
        else *reinterpret_cast<float2*>(p.parts + (int64_t)part * T * p.H + at) = s;
    }
}

// out = the sums of the split workgroups, in their order; eight columns a thread.
__global__ void __launch_bounds__(256)
layer_sum_kernel(LayerArgs p) {
    const int64_t n = p.T * p.H, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= n) return;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int v = 0; v < p.split; ++v) {
        const v4f* a = reinterpret_cast<const v4f*>(p.parts + (int64_t)v * n + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += a[j >> 2][j & 3];
    }
    *reinterpret_cast<uint4*>(p.out + i) =
        make_uint4(bf16x2(s[0], s[1]), bf16x2(s[2], s[3]), bf16x2(s[4], s[5]), bf16x2(s[6], s[7]));
}

template <int WF, int NT>
hipError_t launch_gate_up(const LayerArgs& p, hipStream_t s) {
    // 16 (NT > 1: 8) loads of 16 bytes a lane and group
    constexpr int L = loads_per_step(WF), KS = NT == 1 || L == 4 ? 4 / L : 2 / L < 1 ? 1 : 2 / L;
    const int64_t rows = p.T * p.k, experts = p.E < rows ? p.E : rows;
    const int64_t units = experts * (p.F / 32), fit = 2 * device_cu_count();
    const dim3 grid((unsigned)(units < fit ? units : fit));
    if constexpr (KS > 1)               // (groups of one step are always whole)
        if (p.H / 128 % KS) {
            hipLaunchKernelGGL((layer_gate_up_kernel<WF, NT, KS, false>), grid, dim3(64 * kGuWaves),
                               plan_lds_bytes(p), s, p);
            return hipGetLastError();
        }
    hipLaunchKernelGGL((layer_gate_up_kernel<WF, NT, KS, true>), grid, dim3(64 * kGuWaves),
                       plan_lds_bytes(p), s, p);
    return hipGetLastError();
}

template <int WF, int NT, int RT>
hipError_t launch_down(const LayerArgs& p, hipStream_t s) {
    // 4 loads a lane, tile and group, 2 where the rows' registers need the room
    constexpr int L = loads_per_step(WF), KS = RT * NT >= 8 && L < 4 ? 2 / L : 4 / L;
    const dim3 grid((unsigned)(p.H / (16 * RT) * p.split));
    const size_t lds = down_lds(p.T, p.k, p.E, RT);
    if constexpr (KS > 1)
        if (p.F / 128 % KS) {
            hipLaunchKernelGGL((layer_down_kernel<WF, NT, KS, false, RT>), grid, dim3(64 * kDnWaves), lds, s, p);
            return hipGetLastError();
        }
    hipLaunchKernelGGL((layer_down_kernel<WF, NT, KS, true, RT>), grid, dim3(64 * kDnWaves), lds, s, p);
    return hipGetLastError();
}

// Tiles of 16 rows that a unit takes of an expert: enough for the rows that an
// expert gets with evenly spread tokens and some more (mean + 3 sigma); an expert
// with more rows takes further turns, its weights then coming from the L2.  One
// tile leaves the registers to twice the weights in flight.
int row_tiles(const LayerArgs& p) {
    const int64_t mean = (p.T * p.k + p.E - 1) / p.E;
    return p.T <= 16 || mean <= 8 ? 1 : p.T <= 32 || mean <= 18 ? 2 : 4;
}

template <int WF, int NT>
hipError_t launch_layer_rows(const LayerArgs& p, hipStream_t s) {
    hipError_t e = launch_gate_up<WF, NT>(p, s);
    if (e != hipSuccess) return e;
    const int rt = down_tiles(WF == kBf16, p.T, p.k, p.E);
    if (rt == 1) e = launch_down<WF, NT, 1>(p, s);
    else if (rt == 2) e = launch_down<WF, NT, 2>(p, s);
    else if constexpr (WF != kBf16 && NT < 4) e = launch_down<WF, NT, 4>(p, s);
    else e = hipErrorInvalidValue;      // (four tiles: MX weights, at most 32 tokens, so NT <= 2)
    if (e != hipSuccess || p.split == 1) return e;
    hipLaunchKernelGGL(layer_sum_kernel, dim3((unsigned)((p.T * p.H / 8 + 255) / 256)), dim3(256), 0, s, p);
    return hipGetLastError();
}

template <int WF>
hipError_t launch_layer_fmt(const LayerArgs& p, hipStream_t s) {
    const int nt = row_tiles(p);
    return nt == 1 ? launch_layer_rows<WF, 1>(p, s) : nt == 2 ? launch_layer_rows<WF, 2>(p, s)
                                                              : launch_layer_rows<WF, 4>(p, s);
}

template <int XF, bool ODD>
void launch_few(const LinearArgs& a, int64_t M, hipStream_t s) {
    const int64_t units = (M < a.G ? M : a.G) * ((a.N + kLinRows - 1) / kLinRows);
    const int64_t fit = 2 * device_cu_count();
    const dim3 grid((unsigned)(units < fit ? units : fit));
    auto go = [&](auto nt, auto ks) {
        constexpr int NT = decltype(nt)::value, KS = decltype(ks)::value;
        if (!ODD && a.K / 128 % KS == 0)
            hipLaunchKernelGGL((linear4_few_kernel<XF, NT, KS, !ODD, ODD>), grid, dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((linear4_few_kernel<XF, NT, KS, false, ODD>), grid, dim3(256), 0, s, a);
    };
    // One tile of rows leaves the registers to twice the weights in flight; past 16
    // rows an expert's weights come again for every tile (from the L2).  Measured on
    // 8 x (14336, 4096) with as many rows each, one / four tiles: 8 rows 42.7 / 48.7
    // us, 16 47.4 / 52.5, 24 79.4 / 57.8; on 64 such experts 8 rows 360 / 414, 24 623
    // / 495.  An average of 8 rows leaves few experts with more than 16.
    if (M <= 16 || M <= (int64_t)8 * a.G)
        go(std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
    else go(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
}

}  // namespace

hipError_t launch_linear4_few(bool x_fp4, const uint8_t* x, const uint8_t* xs, const int64_t* offs, int G,
                              int64_t M, const uint8_t* w, const uint8_t* ws, int64_t N, int64_t K,
                              const float* rscale, uint16_t* y, hipStream_t s) {
    const LinearArgs a{x, xs, w, ws, offs, rscale, y, N, K, G};
    const bool odd = K % 128 != 0;
    if (x_fp4) {
        if (odd) launch_few<kFp4, true>(a, M, s);
        else launch_few<kFp4, false>(a, M, s);
    } else {
        if (odd) launch_few<kFp8, true>(a, M, s);
        else launch_few<kFp8, false>(a, M, s);
    }
    return hipGetLastError();
}

int layer_split(bool bf16, int64_t T, int k, int E, int64_t H) {
    const int64_t tiles = H / (16 * down_tiles(bf16, T, k, E)), s = (kSplitFull + tiles - 1) / tiles;
    return (int)(s < 8 ? s : 8);
}

hipError_t launch_layer(LayerWeights wf, const LayerArgs& p, hipStream_t s) {
    const unsigned grid = wf == LayerWeights::kBf16 ? 1u : 1u + (unsigned)p.T;
    hipLaunchKernelGGL(layer_prep_kernel, dim3(grid), dim3(kPrepThreads), prep_lds(p.T, p.E, p.k),
                       s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    switch (wf) {
        case LayerWeights::kBf16: return launch_layer_fmt<few::kBf16>(p, s);
        case LayerWeights::kMxfp8: return launch_layer_fmt<few::kFp8>(p, s);
        case LayerWeights::kMxfp4: return launch_layer_fmt<few::kFp4>(p, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace mx
