// The whole MoE layer for a few tokens with MXFP4 experts. At most 16 tokens
// are the columns of one 16x16x128 MFMA, so every hit expert's weights cross
// HBM once whatever the number of tokens that picked it, and an expert's
// product is taken for all 16 columns at no extra cost; only picked
// (token, expert) pairs are kept. Bound by HBM: 3 H I (1/2 + 1/32) bytes per
// distinct hit expert.
//
//   gate/up: an item is 8 intermediate columns of one expert (8 gate and 8 up
//     rows, one MFMA operand); the 8 waves split K and add their partial sums
//     through LDS. Items are I/8 per hit expert, so with one workgroup per CU
//     the load is even for any number of experts. The quantised tokens stay in
//     registers for the whole kernel.
//   down + combine: a workgroup owns 32 columns of the output for every hit
//     expert; the waves split K, quantise the fp32 intermediate as they read it
//     (a lane holds a whole block of 32, so its largest needs no exchange), and
//     add each expert's product, times its routing weight, in fp32. One rounding
//     at the end, no atomics: the result does not depend on the schedule.
#include "mx_dev.h"

namespace moe {
namespace {

constexpr int kFewT = 16;      // tokens: the columns of one MFMA
constexpr int kFewK = 8;       // picks per token
constexpr int kFewSlots = kFewT * kFewK;
constexpr int kFewThreads = 512;
constexpr int kFewWaves = kFewThreads / 64;
constexpr int kFewMaxE = 1024;
constexpr int kFewSteps = 8;   // K steps of 128 per wave: H <= 8192

struct FewArgs {
    const uint16_t* x;         // [T][H] bf16
    const int32_t* ids;        // [T][k]
    const float* topk_w;       // [T][k]
    int T, k, H, I, base, E_local, has_shared;
    const uint8_t *w13, *w13s, *w2, *w2s, *ws13, *ws13s, *ws2, *ws2s;
    float* a;                  // [T*k + T][I] fp32 intermediate, row = slot (T*k + t: shared)
    uint16_t* out;             // [T][H] bf16
};

// The distinct local experts among the picks, ascending, the shared expert
// behind them; and for each (group, token) the first slot that picked it and
// the sum of the weights of all that did (an id may stand twice in a row).
struct FewMap {
    uint32_t hit[kFewMaxE / 32];
    int ids[kFewSlots];
    int expert[kFewSlots + 1];
    short slot[(kFewSlots + 1) * kFewT];   // -1: not picked
    float weight[(kFewSlots + 1) * kFewT];
    int n;
};

__device__ __forceinline__ int build_few_map(FewMap& m, const FewArgs& p) {
    const int tid = threadIdx.x, S = p.T * p.k;
    for (int i = tid; i < kFewMaxE / 32; i += kFewThreads) m.hit[i] = 0;
    __syncthreads();
    for (int i = tid; i < S; i += kFewThreads) {
        const int id = p.ids[i];  // any value: compared before the subtraction can overflow
        const int e = id >= p.base && id - p.base < p.E_local ? id - p.base : -1;
        m.ids[i] = e;
        if (e >= 0) atomicOr(&m.hit[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    for (int e = tid; e < p.E_local; e += kFewThreads) {
        if (m.hit[e >> 5] >> (e & 31) & 1) {
            int pos = __popc(m.hit[e >> 5] & ((1u << (e & 31)) - 1));
            for (int w = 0; w < e >> 5; ++w) pos += __popc(m.hit[w]);
            m.expert[pos] = e;
        }
    }
    if (tid == 0) {
        int n = 0;
        for (int w = 0; w < kFewMaxE / 32; ++w) n += __popc(m.hit[w]);
        if (p.has_shared) m.expert[n++] = -1;
        m.n = n;
    }
    __syncthreads();
    for (int i = tid; i < m.n * kFewT; i += kFewThreads) {
        const int e = m.expert[i / kFewT], t = i % kFewT;
        int slot = -1;
        float w = 0.f;
        if (t < p.T) {
            if (e < 0) {
                slot = S + t;
                w = 1.0f;
            } else {
                for (int j = p.k - 1; j >= 0; --j)
                    if (m.ids[t * p.k + j] == e) {
                        slot = t * p.k + j;
                        w += p.topk_w[slot];
                    }
            }
        }
        m.slot[i] = (short)slot;
        m.weight[i] = w;
    }
    __syncthreads();
    return m.n;
}

__device__ __forceinline__ f32x4 mfma16_fp4(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
    const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

__global__ __launch_bounds__(kFewThreads) void few_gate_up_kernel(FewArgs p) {
    __shared__ FewMap m;
    __shared__ float red[kFewWaves][16][17];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & 15, lk = lane >> 4;
    const int nk = p.H / 128, ns = (nk + kFewWaves - 1) / kFewWaves;
    const int s0 = wave * ns, s1 = min(nk, s0 + ns);
    const int kb = p.H / kMxBlock;
    const int n = build_few_map(m, p);

    // the tokens, quantised as moe_quantize_mxfp4 does: lane (li, lk) holds
    // token li's block 4 step + lk
    u32x4 b[kFewSteps];
    uint32_t sb[kFewSteps];
#pragma unroll
    for (int q = 0; q < kFewSteps; ++q) {
        b[q] = u32x4{0, 0, 0, 0};
        sb[q] = 127;
        if (s0 + q < s1 && li < p.T) {
            const u32x4* src = reinterpret_cast<const u32x4*>(p.x + (size_t)li * p.H + (4 * (s0 + q) + lk) * kMxBlock);
            float v[32];
            uint32_t mx = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const u32x4 w = src[c];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[8 * c + 2 * i] = bf16_lo(w[i]);
                    v[8 * c + 2 * i + 1] = bf16_hi(w[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) mx = max(mx, abs_bits(v[i]));
            sb[q] = mx_scale_byte(mx);
            const float inv = mx_inverse(sb[q]);
#pragma unroll
            for (int c = 0; c < 4; ++c) b[q][c] = mx_pack8(v + 8 * c, inv);
        }
    }

    const int per = p.I / 8, n_items = n * per;
    for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
        const int g = item / per, i0 = item % per * 8;
        const int e = m.expert[g];
        const uint8_t* W = e < 0 ? p.ws13 : p.w13 + (size_t)e * 2 * p.I * (p.H / 2);
        const uint8_t* Ws = e < 0 ? p.ws13s : p.w13s + (size_t)e * 2 * p.I * kb;
        const int row = i0 + (li & 7) + (li >> 3) * p.I;  // MFMA rows 0..7 gate, 8..15 up
        const uint8_t* wr = W + (size_t)row * (p.H / 2) + 16 * lk;
        const uint8_t* sr = Ws + (size_t)row * kb + lk;
        u32x4 a[kFewSteps];
        uint32_t sa[kFewSteps];
#pragma unroll
        for (int q = 0; q < kFewSteps; ++q)
            if (s0 + q < s1) {
                a[q] = *reinterpret_cast<const u32x4*>(wr + 64 * (s0 + q));
                sa[q] = sr[4 * (s0 + q)];
            }
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < kFewSteps; ++q)
            if (s0 + q < s1) acc = mfma16_fp4(a[q], b[q], acc, sa[q], sb[q]);
        __syncthreads();  // the last item's sums have been read
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][4 * lk + r][li] = acc[r];
        __syncthreads();
        if (threadIdx.x < 8 * kFewT) {
            const int i = threadIdx.x & 7, t = threadIdx.x >> 3;
            const int slot = m.slot[g * kFewT + t];
            if (slot >= 0) {
                float gs = 0.f, us = 0.f;
#pragma unroll
                for (int w = 0; w < kFewWaves; ++w) {
                    gs += red[w][i][t];
                    us += red[w][8 + i][t];
                }
                p.a[(size_t)slot * p.I + i0 + i] = silu_mul(gs, us);
            }
        }
    }
}

constexpr int kFewCols = 32;  // output columns per workgroup of the down kernel

__global__ __launch_bounds__(kFewThreads) void few_down_kernel(FewArgs p) {
    __shared__ FewMap m;
    __shared__ float red[kFewWaves][kFewCols][17];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane & 15, lk = lane >> 4;
    const int nk = p.I / 128, kb = p.I / kMxBlock;
    const int h0 = blockIdx.x * kFewCols;
    const int n = build_few_map(m, p);
    f32x4 total[2] = {};
    for (int g = 0; g < n; ++g) {
        const int e = m.expert[g];
        const uint8_t* W = (e < 0 ? p.ws2 : p.w2 + (size_t)e * p.H * (p.I / 2)) + (size_t)(h0 + li) * (p.I / 2) + 16 * lk;
        const uint8_t* Ws = (e < 0 ? p.ws2s : p.w2s + (size_t)e * p.H * kb) + (size_t)(h0 + li) * kb + lk;
        const int slot = m.slot[g * kFewT + li];
        const float* ar = p.a + (size_t)max(slot, 0) * p.I + lk * kMxBlock;
        f32x4 acc[2] = {};
        for (int s = wave; s < nk; s += kFewWaves) {
            u32x4 b = {0, 0, 0, 0};
            uint32_t sb = 127;
            if (slot >= 0) {
                float v[32];
                uint32_t mx = 0;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const f32x4 q = *reinterpret_cast<const f32x4*>(ar + 128 * s + 4 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[4 * c + i] = q[i];
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) mx = max(mx, abs_bits(v[i]));
                sb = mx_scale_byte(mx);
                const float inv = mx_inverse(sb);
#pragma unroll
                for (int c = 0; c < 4; ++c) b[c] = mx_pack8(v + 8 * c, inv);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const u32x4 a = *reinterpret_cast<const u32x4*>(W + (size_t)16 * q * (p.I / 2) + 64 * s);
                const uint32_t sa = Ws[(size_t)16 * q * kb + 4 * s];
                acc[q] = mfma16_fp4(a, b, acc[q], sa, sb);
            }
        }
        // a token that did not pick this expert takes nothing from it, not even a NaN
        const float w = m.weight[g * kFewT + li];
        if (slot >= 0) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int r = 0; r < 4; ++r) total[q][r] = __builtin_fmaf(w, acc[q][r], total[q][r]);
        }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][16 * q + 4 * lk + r][li] = total[q][r];
    __syncthreads();
    const int c = threadIdx.x & 31, t = threadIdx.x >> 5;
    if (t < p.T) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) s += red[w][c][t];
        p.out[(size_t)t * p.H + h0 + c] = (uint16_t)f32_to_bf16_bits(s);
    }
}

struct FewWs {
    uint32_t* sync;
    float* logits;
    float* a;
    size_t bytes;
};

FewWs carve_few(const moe_expert_weights* w, int T, int E, int k, void* base) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = align_up(off + bytes, 256);
        return base ? (void*)((uint8_t*)base + o) : nullptr;
    };
    FewWs r{};
    r.sync = (uint32_t*)take(256);
    r.logits = (float*)take((size_t)T * E * 4);
    r.a = (float*)take(((size_t)T * k + T) * w->I * 4);
    r.bytes = off;
    return r;
}

}  // namespace

size_t layer_few_workspace_bytes(const moe_expert_weights* w, int T, int E, int k) {
    return carve_few(w, T, E, k, nullptr).bytes;
}

moe_status launch_layer_few(const void* x, const void* w_router, const float* bias, int T, int E, int k,
                            int scoring, int renorm, const moe_expert_weights* w, int base, int32_t* topk_ids,
                            float* topk_w, void* out, void* ws, hipStream_t st) {
    const FewWs s = carve_few(w, T, E, k, ws);
    if (w_router) {
        const moe_status r = launch_route(x, w_router, bias, MOE_BF16, T, w->H, E, k, scoring, renorm, s.logits,
                                          topk_ids, topk_w, st);
        if (r) return r;
    }
    FewArgs p{};
    p.x = (const uint16_t*)x;
    p.ids = topk_ids;
    p.topk_w = topk_w;
    p.T = T;
    p.k = k;
    p.H = w->H;
    p.I = w->I;
    p.base = base;
    p.E_local = w->E_local;
    p.has_shared = w->ws13 != nullptr;
    p.w13 = (const uint8_t*)w->w13;
    p.w13s = (const uint8_t*)w->w13_scale;
    p.w2 = (const uint8_t*)w->w2;
    p.w2s = (const uint8_t*)w->w2_scale;
    p.ws13 = (const uint8_t*)w->ws13;
    p.ws13s = (const uint8_t*)w->ws13_scale;
    p.ws2 = (const uint8_t*)w->ws2;
    p.ws2s = (const uint8_t*)w->ws2_scale;
    p.a = s.a;
    p.out = (uint16_t*)out;
    hipLaunchKernelGGL(few_gate_up_kernel, dim3(device_info().cu_count), dim3(kFewThreads), 0, st, p);
    const moe_status r = check_launch("few_gate_up_kernel");
    if (r) return r;
    hipLaunchKernelGGL(few_down_kernel, dim3(w->H / kFewCols), dim3(kFewThreads), 0, st, p);
    return check_launch("few_down_kernel");
}

}  // namespace moe
