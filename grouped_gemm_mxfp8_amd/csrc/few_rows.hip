// GroupedLinear on MXFP4 weights for few rows an expert, and the whole MoE
// layer for a few tokens (gfx950).  Both stream the weights once through the
// core in few_rows.h.
//
// The layer runs as three launches on one stream:
//  * layer_prep: workgroup 0 routes (top-k by a bitwise search for the k-th
//    largest key, softmax of the selected logits) and lists the routed rows
//    sorted by (expert, token); the other workgroups quantize one token of x
//    each to MXFP8 (MX weights only).
//  * layer_gate_up: a workgroup takes 32 columns of F of one routed expert (64
//    rows of W1), its four waves a quarter of H each; z = r silu(a) b leaves
//    as MXFP8 blocks (MX weights) or bf16.
//  * layer_down: a workgroup takes 16 rows of every routed expert's W2 and adds
//    the experts' products in fp32 in LDS, so the combine needs no atomics, no
//    second pass and has one fixed order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "few_rows.h"
#include "internal.h"
#include "mx_device.h"

namespace mx {
namespace {

using namespace few;

// ---- GroupedLinear, few rows an expert --------------------------------------

constexpr int kLinRows = 64;      // rows of W (columns of y) per workgroup
constexpr int kLinWaves = 4;

struct LinearArgs {
    const uint8_t *x, *xs, *w, *ws;
    const int64_t* offs;
    const float* rscale;
    uint16_t* y;
    int64_t N, K;
};

// One chunk of up to 16 NT rows [m0, m0 + rows) of expert e: y[.., n0 .. n0+63].
template <int XF, int NT, bool ODD>
__device__ __forceinline__ void linear_chunk(const LinearArgs& p, int e, int64_t n0, int64_t m0, int rows,
                                             float* part, int wave, int lane) {
    const int q = lane >> 4, r16 = lane & 15;
    Row w[4], x[NT];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        // tiles past N (N % 32 == 0) repeat the first one and are not stored
        const int64_t n = n0 + 16 * t < p.N ? n0 + 16 * t : n0;
        w[t] = row_of<kFp4>(p.w, p.ws, (int64_t)e * p.N + n + r16, p.K, lane);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
        x[n] = row_of<XF>(p.x, p.xs, m0 + min(n * 16 + r16, rows - 1), p.K, lane);
    v4f acc[4][NT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[t][n] = v4f{0.f, 0.f, 0.f, 0.f};
    const int steps = (int)((p.K + 127) / 128);
    const int s0 = uni(wave * steps / kLinWaves), s1 = uni((wave + 1) * steps / kLinWaves);
    mac_rows<kFp4, XF, 4, NT, 4, ODD>(acc, w, x, s0, s1, p.K, q);
    // the waves' K parts, added in wave order; thread (token, 4 columns)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (n * 16 >= rows) break;
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 4; ++t)
            *reinterpret_cast<v4f*>(part + ((wave * 4 + t) * 64 + lane) * 4) = acc[t][n];
        __syncthreads();
        const int tid = wave * 64 + lane;
        const int tok = tid >> 4, c4 = tid & 15;          // columns n0 + 4 c4 .. + 3
        const int at = ((c4 >> 2) * 64 + (c4 & 3) * 16 + tok) * 4;
        v4f s = *reinterpret_cast<const v4f*>(part + at);
#pragma unroll
        for (int v = 1; v < kLinWaves; ++v) s += *reinterpret_cast<const v4f*>(part + v * 1024 + at);
        const int row = n * 16 + tok;
        const int64_t col = n0 + 4 * c4;
        if (row < rows && col < p.N) {
            const float f = p.rscale ? p.rscale[m0 + row] : 1.0f;
            *reinterpret_cast<uint2*>(p.y + (m0 + row) * p.N + col) =
                make_uint2(bf16x2(s[0] * f, s[1] * f), bf16x2(s[2] * f, s[3] * f));
        }
    }
}

template <int XF, int NTMAX, bool ODD>
__global__ void __launch_bounds__(256)
linear4_few_kernel(LinearArgs p) {
    __shared__ __attribute__((aligned(16))) float part[kLinWaves * 1024];
    const int e = blockIdx.y;
    const int64_t lo = p.offs[e], hi = p.offs[e + 1];
    const int wave = uni(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t n0 = (int64_t)blockIdx.x * kLinRows;
    for (int64_t m0 = lo; m0 < hi; m0 += 16 * NTMAX) {
        const int rows = uni((int)min((int64_t)(16 * NTMAX), hi - m0));
        if (NTMAX > 1 && rows > 16) {
            if (NTMAX > 2 && rows > 32) linear_chunk<XF, NTMAX, ODD>(p, e, n0, m0, rows, part, wave, lane);
            else linear_chunk<XF, NTMAX < 2 ? NTMAX : 2, ODD>(p, e, n0, m0, rows, part, wave, lane);
        } else {
            linear_chunk<XF, 1, ODD>(p, e, n0, m0, rows, part, wave, lane);
        }
    }
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

// Workgroup 0 of layer_prep.  LDS: the selected experts of each token as bits,
// each expert's rows, and each token's softmax terms.  W: 64-expert words per
// token that the registers hold (1 for E <= 64, else the largest).
template <int W>
__device__ void layer_plan(const float* __restrict__ logits, int T, int E, int k, const LayerPlan& plan,
                           uint8_t* smem) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int words = (E + 63) / 64;                                     // 64-expert words per token
    uint64_t* sel = reinterpret_cast<uint64_t*>(smem);                   // [T][words]
    int* cnt = reinterpret_cast<int*>(sel + (int64_t)T * words);         // [E] rows, then first rows
    float* mx = reinterpret_cast<float*>(cnt + E);                       // [T] largest logit
    float* inv = mx + T;                                                 // [T] 1 / sum of exponentials
    for (int t = wave; t < T; t += kPrepThreads / 64) {
        uint32_t key[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int e = lane + 64 * i;
            key[i] = e < E ? logit_key(logits[(int64_t)t * E + e]) : 0u;
        }
        // th: the largest value that at least k keys reach (0 if fewer routed)
        uint32_t th = 0;
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t cand = th | (1u << bit);
            int n = 0;
#pragma unroll
            for (int i = 0; i < W; ++i) n += __popcll(__ballot(key[i] >= cand));
            if (n >= k) th = cand;
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
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
        const float m = key_logit(top);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (on[i]) sum += expf(key_logit(key[i]) - m);
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
        if (lane < words) sel[t * words + lane] = mine;
        if (lane == 0) {
            mx[t] = m;
            inv[t] = 1.0f / sum;
        }
    }
    __syncthreads();
    // rows of each expert
    for (int e = tid; e < E; e += kPrepThreads) {
        int n = 0;
        for (int t = 0; t < T; ++t) n += (int)(sel[t * words + (e >> 6)] >> (e & 63) & 1);
        cnt[e] = n;
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
    // (token, expert) pairs to their rows: tokens ascend within an expert
    for (int i = tid; i < T * E; i += kPrepThreads) {
        const int t = i / E, e = i - t * E;
        const int wd = e >> 6, sh = e & 63;
        if (!(sel[t * words + wd] >> sh & 1)) continue;
        int before = 0;
        for (int u = 0; u < t; ++u) before += (int)(sel[u * words + wd] >> sh & 1);
        const int row = cnt[e] + before;
        plan.tok[row] = t;
        const float v = key_logit(logit_key(logits[(int64_t)t * E + e]));
        plan.r[row] = expf(v - mx[t]) * inv[t];
    }
}

size_t plan_lds(int64_t T, int E) {
    return (size_t)(T * ((E + 63) / 64) * 8 + E * 4 + T * 8);
}

// MXFP8 blocks of one token (H % 128 == 0), as mxfp8_quantize makes them; a
// block with an infinity or a NaN gets the NaN scale, so that the token's
// output says so.
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
        if (bad) o = make_uint2(0u, 0u);
        *reinterpret_cast<uint2*>(codes + u * 8) = o;
        if ((threadIdx.x & 3) == 0) scales[u >> 2] = bad ? 255 : (uint8_t)c;
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

// Rows [c0, c0 + rows) of the expert's list, columns f0 .. f0 + 31 of z.
template <int WF, int NT>
__device__ __forceinline__ void gate_up_chunk(const LayerArgs& p, int e, int row0, int rows, int64_t f0,
                                              float* part, int wave, int lane) {
    constexpr int XF = WF == kBf16 ? kBf16 : kFp8;
    const int q = lane >> 4, r16 = lane & 15;
    Row w[4], x[NT];
#pragma unroll
    for (int t = 0; t < 4; ++t)      // tiles 0, 1: gate rows; 2, 3: up rows
        w[t] = row_of<WF>(p.w1, p.w1s, (int64_t)e * 2 * p.F + (t >> 1) * p.F + f0 + (t & 1) * 16 + r16, p.H,
                          lane);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int tok = p.plan.tok[row0 + min(n * 16 + r16, rows - 1)];
        x[n] = row_of<XF>(WF == kBf16 ? reinterpret_cast<const uint8_t*>(p.x) : p.xq, p.xqs, tok, p.H, lane);
    }
    v4f acc[4][NT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[t][n] = v4f{0.f, 0.f, 0.f, 0.f};
    const int steps = (int)(p.H / 128);
    const int s0 = uni(wave * steps / kGuWaves), s1 = uni((wave + 1) * steps / kGuWaves);
    mac_rows<WF, XF, 4, NT, 4 / loads_per_step(WF), false>(acc, w, x, s0, s1, p.H, q);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (n * 16 >= rows) break;
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 4; ++t)
            *reinterpret_cast<v4f*>(part + ((wave * 4 + t) * 64 + lane) * 4) = acc[t][n];
        __syncthreads();
        // thread (token, two columns f0 + 2 c, + 1): the 16 threads of a token
        // are one DPP row and hold one block of 32
        const int tid = wave * 64 + lane;
        const int tok = tid >> 4, c = (tid & 15) * 2;
        const int at = ((c >> 4) * 64 + ((c & 15) >> 2) * 16 + tok) * 4 + (c & 3);
        float g[2] = {0.f, 0.f}, u[2] = {0.f, 0.f};
#pragma unroll
        for (int v = 0; v < kGuWaves; ++v) {
            const float2 a = *reinterpret_cast<const float2*>(part + v * 1024 + at);
            const float2 b = *reinterpret_cast<const float2*>(part + v * 1024 + 512 + at);
            g[0] += a.x;
            g[1] += a.y;
            u[0] += b.x;
            u[1] += b.y;
        }
        const int row = n * 16 + tok;
        const bool live = row < rows;
        const float r = live ? p.plan.r[row0 + row] : 0.f;
        float z[2];
#pragma unroll
        for (int v = 0; v < 2; ++v)
            z[v] = r * (g[v] * __builtin_amdgcn_rcpf(1.0f + __expf(-g[v])) * u[v]);
        const int64_t zrow = row0 + row;
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
            const uint32_t sc = bad ? 255u : scale_code_from_amax_bits(m);
            const uint32_t o = bad ? 0u : e4m3x2_scaled(0u, z[0], z[1], e4m3_limit_from_code(sc),
                                                        scale_from_code(sc), false);
            if (live) {
                *reinterpret_cast<uint16_t*>(p.z + zrow * p.F + f0 + c) = (uint16_t)o;
                if (c == 0) p.zs[zrow * (p.F / 32) + f0 / 32] = (uint8_t)sc;
            }
        }
    }
}

template <int WF, int NTMAX>
__global__ void __launch_bounds__(256)
layer_gate_up_kernel(LayerArgs p) {
    __shared__ __attribute__((aligned(16))) float part[kGuWaves * 1024];
    if ((int)blockIdx.y >= *p.plan.n_act) return;
    const int4 a = p.plan.act[blockIdx.y];
    const int e = uni(a.x), first = uni(a.y), count = uni(a.z);
    const int wave = uni(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t f0 = (int64_t)blockIdx.x * 32;
    for (int c0 = 0; c0 < count; c0 += 16 * NTMAX) {
        const int rows = min(16 * NTMAX, count - c0);
        if (NTMAX > 1 && rows > 16) {
            if (NTMAX > 2 && rows > 32) gate_up_chunk<WF, NTMAX>(p, e, first + c0, rows, f0, part, wave, lane);
            else gate_up_chunk<WF, NTMAX < 2 ? NTMAX : 2>(p, e, first + c0, rows, f0, part, wave, lane);
        } else {
            gate_up_chunk<WF, 1>(p, e, first + c0, rows, f0, part, wave, lane);
        }
    }
}

// ---- the layer: down and combine -------------------------------------------------

constexpr int kDnWaves = 8;

// z rows [row0, row0 + rows) against rows h0 .. h0 + 15 of expert e's W2 over
// the steps [s0, s1): added to the wave's sums out[token][16].
template <int WF, int NT>
__device__ __forceinline__ void down_unit(const LayerArgs& p, int e, int row0, int rows, int64_t h0, int s0,
                                          int s1, float* out, int lane) {
    constexpr int XF = WF == kBf16 ? kBf16 : kFp8;
    const int q = lane >> 4, r16 = lane & 15;
    Row w[1], x[NT];
    w[0] = row_of<WF>(p.w2, p.w2s, (int64_t)e * p.H + h0 + r16, p.F, lane);
#pragma unroll
    for (int n = 0; n < NT; ++n)
        x[n] = row_of<XF>(p.z, p.zs, row0 + min(n * 16 + r16, rows - 1), p.F, lane);
    v4f acc[1][NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[0][n] = v4f{0.f, 0.f, 0.f, 0.f};
    mac_rows<WF, XF, 1, NT, 8 / loads_per_step(WF), false>(acc, w, x, s0, s1, p.F, q);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int row = n * 16 + r16;
        if (row < rows) {       // an expert's tokens are distinct: no two lanes share a sum
            v4f* o = reinterpret_cast<v4f*>(out + p.plan.tok[row0 + row] * 16 + 4 * q);
            *o += acc[0][n];
        }
    }
}

// TMAX: bound of T that sizes the sums in LDS.
template <int WF, int NTMAX, int TMAX>
__global__ void __launch_bounds__(64 * kDnWaves)
layer_down_kernel(LayerArgs p) {
    __shared__ __attribute__((aligned(16))) float sums[kDnWaves * TMAX * 16];
    const int tid = threadIdx.x, wave = uni(tid >> 6), lane = tid & 63;
    const int64_t h0 = (int64_t)blockIdx.x * 16;
    const int T = (int)p.T;
    float* out = sums + wave * TMAX * 16;
    for (int i = lane; i < T * 4; i += 64) reinterpret_cast<v4f*>(out)[i] = v4f{0.f, 0.f, 0.f, 0.f};
    const int n_act = uni(*p.plan.n_act);
    const int steps = (int)(p.F / 128);
    // K parts per expert, so that every wave has work with few experts
    const int parts = uni(max(1, min(steps / 4, (2 * kDnWaves + n_act - 1) / max(n_act, 1))));
    for (int u = wave; u < n_act * parts; u += kDnWaves) {
        const int a = u / parts, c = u - a * parts;
        const int4 ex = p.plan.act[a];
        const int e = uni(ex.x), first = uni(ex.y), count = uni(ex.z);
        const int s0 = uni(c * steps / parts), s1 = uni((c + 1) * steps / parts);
        for (int c0 = 0; c0 < count; c0 += 16 * NTMAX) {
            const int rows = min(16 * NTMAX, count - c0);
            if (NTMAX > 1 && rows > 16) {
                if (NTMAX > 2 && rows > 32) down_unit<WF, NTMAX>(p, e, first + c0, rows, h0, s0, s1, out, lane);
                else down_unit<WF, NTMAX < 2 ? NTMAX : 2>(p, e, first + c0, rows, h0, s0, s1, out, lane);
            } else {
                down_unit<WF, 1>(p, e, first + c0, rows, h0, s0, s1, out, lane);
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < T * 8; i += 64 * kDnWaves) {        // two rows of out a thread
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < kDnWaves; ++v) {
            const float2 a = *reinterpret_cast<const float2*>(sums + v * TMAX * 16 + 2 * i);
            s.x += a.x;
            s.y += a.y;
        }
        *reinterpret_cast<uint32_t*>(p.out + (int64_t)(i >> 3) * p.H + h0 + 2 * (i & 7)) = bf16x2(s.x, s.y);
    }
}

template <int WF>
hipError_t launch_layer_fmt(const LayerArgs& p, hipStream_t s) {
    const dim3 gu((unsigned)(p.F / 32), (unsigned)(p.E < p.T * p.k ? p.E : p.T * p.k));
    const dim3 dn((unsigned)(p.H / 16));
    if (p.T <= 16) hipLaunchKernelGGL((layer_gate_up_kernel<WF, 1>), gu, dim3(256), 0, s, p);
    else if (p.T <= 32) hipLaunchKernelGGL((layer_gate_up_kernel<WF, 2>), gu, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((layer_gate_up_kernel<WF, 4>), gu, dim3(256), 0, s, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.T <= 16) hipLaunchKernelGGL((layer_down_kernel<WF, 1, 16>), dn, dim3(64 * kDnWaves), 0, s, p);
    else if (p.T <= 32) hipLaunchKernelGGL((layer_down_kernel<WF, 2, 32>), dn, dim3(64 * kDnWaves), 0, s, p);
    else hipLaunchKernelGGL((layer_down_kernel<WF, 4, kLayerMaxTokens>), dn, dim3(64 * kDnWaves), 0, s, p);
    return hipGetLastError();
}

template <int XF, bool ODD>
void launch_few(const LinearArgs& a, dim3 grid, int64_t M, hipStream_t s) {
    if (M <= 16) hipLaunchKernelGGL((linear4_few_kernel<XF, 1, ODD>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((linear4_few_kernel<XF, 4, ODD>), grid, dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_linear4_few(bool x_fp4, const uint8_t* x, const uint8_t* xs, const int64_t* offs, int G,
                              int64_t M, const uint8_t* w, const uint8_t* ws, int64_t N, int64_t K,
                              const float* rscale, uint16_t* y, hipStream_t s) {
    const LinearArgs a{x, xs, w, ws, offs, rscale, y, N, K};
    const dim3 grid((unsigned)((N + kLinRows - 1) / kLinRows), (unsigned)G);
    const bool odd = K % 128 != 0;
    if (x_fp4) {
        if (odd) launch_few<kFp4, true>(a, grid, M, s);
        else launch_few<kFp4, false>(a, grid, M, s);
    } else {
        if (odd) launch_few<kFp8, true>(a, grid, M, s);
        else launch_few<kFp8, false>(a, grid, M, s);
    }
    return hipGetLastError();
}

hipError_t launch_layer(LayerWeights wf, const LayerArgs& p, hipStream_t s) {
    const unsigned grid = wf == LayerWeights::kBf16 ? 1u : 1u + (unsigned)p.T;
    hipLaunchKernelGGL(layer_prep_kernel, dim3(grid), dim3(kPrepThreads), plan_lds(p.T, p.E), s, p);
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
