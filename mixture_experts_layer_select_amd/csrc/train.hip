// What training the layer needs beside the grouped products: the gated units
// and their gradient, dropout from a counter, and the gradients of the combine
// and of the gate. One pass over the data each, sums in fp32 in a fixed order.
#include "combine_dev.h"

namespace moe {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) v += __shfl_xor(v, s);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) v = fmaxf(v, __shfl_xor(v, s));
    return v;
}

// ============================================================================ dropout
// The random numbers come from Philox4x32-10 (J. Salmon et al., "Parallel
// random numbers: as easy as 1, 2, 3", 2011): a block of four words is a
// function of a 64-bit key and a 128-bit counter. Key: the seed; counter: the
// block's number and the offset. Element i uses 16 bits, half i % 8 of block
// i / 8, so eight neighbours (16 bytes of bf16) cost one block: ten rounds of
// two 32 x 32 -> 64 bit products. With 32 bits an element the products alone would take
// longer than HBM needs for a bf16 element; p is therefore held in units of 2^-16.
struct Dropout {
    const uint64_t* rng;  // device: seed, offset
    uint32_t threshold;   // an element goes where its 16 bits are below; 0: no dropout, rng unread
    float scale;          // 65536 / (65536 - threshold)
};

__device__ __forceinline__ u32x4 philox(uint64_t seed, uint64_t offset, uint64_t block) {
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

// bit j: element i + j stays. kWhole: i is a multiple of eight.
template <bool kWhole>
__device__ __forceinline__ uint32_t keep8(const Dropout& d, uint64_t seed, uint64_t offset, uint64_t i) {
    auto bits = [&](uint64_t block) {
        const u32x4 w = philox(seed, offset, block);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m |= ((w[j] & 0xffffu) >= d.threshold ? 1u : 0u) << (2 * j);
            m |= ((w[j] >> 16) >= d.threshold ? 1u : 0u) << (2 * j + 1);
        }
        return m;
    };
    if constexpr (kWhole) return bits(i >> 3);
    const int s = (int)(i & 7);
    const uint32_t lo = bits(i >> 3);
    return s ? (lo | bits((i >> 3) + 1) << 8) >> s : lo;
}

// out = residual + drop(x), flat. The outputs may be the inputs: a thread reads its eight elements before it writes
// them.
template <typename T, bool kVec>
__global__ __launch_bounds__(256) void dropout_kernel(const T* x, const T* residual, long n, Dropout d, T* out) {
    uint64_t seed = 0, offset = 0;
    if (d.threshold) {
        seed = d.rng[0];
        offset = d.rng[1];
    }
    for (long i = ((long)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (long)gridDim.x * 256 * 8) {
        const int m = (int)min(8L, n - i);
        float v[8], r[8] = {};
        if (kVec && m == 8) {
            get8<true>(x + i, 0, 8, v);
            if (residual) get8<true>(residual + i, 0, 8, r);
        } else {
            get8<false>(x + i, 0, m, v);
            if (residual) get8<false>(residual + i, 0, m, r);
        }
        const uint32_t keep = d.threshold ? keep8<true>(d, seed, offset, (uint64_t)i) : 0xffu;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = r[j] + (keep >> j & 1 ? v[j] * d.scale : 0.f);
        if (kVec && m == 8) put8<true>(out + i, 0, 8, v);
        else put8<false>(out + i, 0, m, v);
    }
}

// ============================================================================ gated units
// gu holds a row's gate columns G and, behind them, its up columns U:
//   a = drop(silu(G) U),  silu(G) = G s,  s = 1 / (1 + exp(-G))
//   da' = drop(da),  dU = da' silu(G),  dG = da' U s (1 + G (1 - s))
// A thread takes eight columns of a row. fp32 has expf, whose last bits it holds. a and the gradients may be written
// over the inputs: a thread reads all its elements before it writes.
__device__ __forceinline__ float exp_for(float v, float) { return expf(v); }
__device__ __forceinline__ float exp_for(float v, uint16_t) { return __expf(v); }

template <typename T, bool kVec, bool kGrad>
__global__ __launch_bounds__(256) void swiglu_kernel(const T* gu, const T* da, const int32_t* n_rows, int max_rows,
                                                     int I, Dropout d, T* dgu, T* a) {
    const int rows = n_rows ? max(0, min(*n_rows, max_rows)) : max_rows;
    const int chunks = (I + 7) / 8;
    const long n = (long)rows * chunks;
    uint64_t seed = 0, offset = 0;
    if (d.threshold) {
        seed = d.rng[0];
        offset = d.rng[1];
    }
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) {
        const long row = i / chunks;
        const int c = (int)(i - row * chunks) * 8;
        const size_t at = (size_t)row * I;
        float g[8], u[8], t[8];
        get8<kVec>(gu + 2 * at, c, I, g);
        get8<kVec>(gu + 2 * at + I, c, I, u);
        if (kGrad) get8<kVec>(da + at, c, I, t);
        const uint32_t keep = d.threshold ? keep8<kVec>(d, seed, offset, (uint64_t)at + c) : 0xffu;
        float av[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool on = keep >> j & 1;
            const float s = 1.0f / (1.0f + exp_for(-g[j], T{}));
            const float silu = g[j] * s;
            av[j] = on ? silu * u[j] * d.scale : 0.f;
            if (kGrad) {
                const float w = on ? t[j] * d.scale : 0.f;
                const float dg = w * u[j] * (s * (1.0f + g[j] * (1.0f - s)));
                u[j] = on ? w * silu : 0.f;
                g[j] = on ? dg : 0.f;
            }
        }
        if (kGrad) {
            put8<kVec>(dgu + 2 * at, c, I, g);
            put8<kVec>(dgu + 2 * at + I, c, I, u);
        }
        if (!kGrad || a) put8<kVec>(a + at, c, I, av);
    }
}

// ============================================================================ gradient of the combine
// out[t] = sum_j w[t,j] y[row(t,j)] + y[shared row t]:
//   dy[row(t,j)] = w[t,j] dout[t],  dy[shared row t] = dout[t],  dw[t,j] = <dout[t], y[row(t,j)]>
// A workgroup takes the picks [blockIdx.y per, + per) of a token, at most kPicks; the last one takes the shared row
// too. dy may be y: a row belongs to one pick, and a thread reads its columns before it writes them.
constexpr int kPicks = 8;
struct CombineGrad {
    const void *dout, *y;
    const int32_t* slot_to_row;
    const float* topk_w;
    int t0, T, k, H;
    const int32_t* offsets;
    int shared_group, per;  // picks of a workgroup
    void* dy;
    float* dw;  // null: y unread
};

// Columns c * 2048 + 8 tid + [0, 8) of the token's row stay in registers for all its picks. kChunks 0: H past the
// registers, dout read anew for each pick.
template <typename T, bool kVec, int kChunks>
__global__ __launch_bounds__(256) void combine_grad_kernel(CombineGrad p) {
    __shared__ float red[4][kPicks];
    const int t = p.t0 + (int)blockIdx.x, H = p.H;
    const T* d = (const T*)p.dout + (size_t)t * H;
    const int j0 = blockIdx.y * p.per, n = min(p.k - j0, p.per);
    const size_t slot = (size_t)t * p.k + j0;
    constexpr int kHold = kChunks ? kChunks : 1;
    float v[kHold][8];
    if constexpr (kChunks > 0) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int h = (c * 256 + threadIdx.x) * 8;
            if (h < H) get8<kVec>(d, h, H, v[c]);
        }
    }
    float sum[kPicks];
#pragma unroll
    for (int j = 0; j < kPicks; ++j) {
        sum[j] = 0.f;
        const int row = j < n ? p.slot_to_row[slot + j] : -1;
        if (row < 0) continue;
        const float w = p.topk_w[slot + j];
        const T* y = (const T*)p.y + (size_t)row * H;
        T* dy = (T*)p.dy + (size_t)row * H;
        auto chunk = [&](int h, const float* x) {
            float o[8];
            if (p.dw) {
                get8<kVec>(y, h, H, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[j] = __builtin_fmaf(x[i], o[i], sum[j]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = x[i] * w;
            put8<kVec>(dy, h, H, o);
        };
        if constexpr (kChunks > 0) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int h = (c * 256 + threadIdx.x) * 8;
                if (h < H) chunk(h, v[c]);
            }
        } else {
            for (int h = threadIdx.x * 8; h < H; h += 256 * 8) {
                get8<kVec>(d, h, H, v[0]);
                chunk(h, v[0]);
            }
        }
    }
    if (p.shared_group >= 0 && blockIdx.y + 1 == gridDim.y) {
        T* dy = (T*)p.dy + (size_t)(p.offsets[p.shared_group] + t) * H;
        if constexpr (kChunks > 0) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int h = (c * 256 + threadIdx.x) * 8;
                if (h < H) put8<kVec>(dy, h, H, v[c]);
            }
        } else {
            for (int h = threadIdx.x * 8; h < H; h += 256 * 8) {
                get8<kVec>(d, h, H, v[0]);
                put8<kVec>(dy, h, H, v[0]);
            }
        }
    }
    if (p.dw) {
#pragma unroll
        for (int j = 0; j < kPicks; ++j) {
            if (j >= n) continue;
            sum[j] = wave_sum(sum[j]);
            if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6][j] = sum[j];
        }
        __syncthreads();
        const int j = threadIdx.x;
        if (j < n) p.dw[slot + j] = red[0][j] + red[1][j] + red[2][j] + red[3][j];
    }
}

// ============================================================================ gradient of the gate
// One wave per token. With D = sum_i w_i dw_i over the picks (of the finished weights, so that a single renormalised
// pick's gradient is exactly 0):
//   sigmoid, renormalised: w_j = s_j / sum s   dl_j = w_j (1 - s_j) (dw_j - D)
//   sigmoid:               w_j = s_j           dl_j = s_j (1 - s_j) dw_j
//   softmax, renormalised: over the picks      dl_j = w_j (dw_j - D)
//   softmax:               over all E          dl_e = [e picked] w_e dw_e - p_e D
// 1 - s is made from exp(-|l|) beside s, not from s: picks are confident, and the fp32 difference is off by 0.9% at a
// logit of 12 and 0 at 18.
// Lane l owns experts 4l .. 4l + 3 of the output row and every 64th pick. An
// expert picked twice gets both picks' sums.
constexpr int kGateMaxE = 256;

struct Sigmoid {
    float s, rest;  // 1 / (1 + exp(-l)) and 1 / (1 + exp(l)), each to a few units of its own last place
};
__device__ __forceinline__ Sigmoid sigmoid_of(float l) {
    const float e = expf(-fabsf(l)), large = 1.0f / (1.0f + e), small = e * large;
    return l >= 0.f ? Sigmoid{large, small} : Sigmoid{small, large};
}

template <typename TO, bool kSigmoid, bool kRenorm>
__global__ __launch_bounds__(256) void route_grad_kernel(const float* __restrict__ logits,
                                                         const int32_t* __restrict__ ids,
                                                         const float* __restrict__ dtopk_w, int T, int E, int k,
                                                         TO* __restrict__ dlogits) {
    const int lane = threadIdx.x & 63;
    const long t = (long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    constexpr int kMax = kGateMaxE / 64;  // picks of a lane
    int id[kMax];
    float l[kMax], dw[kMax], w[kMax];
#pragma unroll
    for (int i = 0; i < kMax; ++i) {
        const int j = lane + 64 * i;
        id[i] = j < k ? ids[t * k + j] : -1;
        dw[i] = j < k ? dtopk_w[t * k + j] : 0.f;
        if ((unsigned)id[i] >= (unsigned)E) id[i] = -1;  // no expert: no part in any sum
        l[i] = id[i] >= 0 ? logits[t * E + id[i]] : 0.f;
        if (id[i] < 0) dw[i] = 0.f;
    }
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, d[kMax];
    if constexpr (kSigmoid) {
        float sum = 0.f, dot = 0.f, rest[kMax];
#pragma unroll
        for (int i = 0; i < kMax; ++i) {
            const Sigmoid s = sigmoid_of(l[i]);
            w[i] = id[i] >= 0 ? s.s : 0.f;
            rest[i] = s.rest;
            sum += w[i];
        }
        sum = kRenorm ? wave_sum(sum) : 1.0f;
#pragma unroll
        for (int i = 0; i < kMax; ++i) dot += w[i] / sum * dw[i];
        dot = kRenorm ? wave_sum(dot) : 0.f;
#pragma unroll
        for (int i = 0; i < kMax; ++i) d[i] = w[i] / sum * rest[i] * (dw[i] - dot);
    } else {
        float all[4], top = -__builtin_inff(), sum = 0.f, dot = 0.f;
        if constexpr (kRenorm) {
#pragma unroll
            for (int i = 0; i < kMax; ++i) top = fmaxf(top, id[i] >= 0 ? l[i] : -__builtin_inff());
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                all[i] = 4 * lane + i < E ? logits[t * E + 4 * lane + i] : -__builtin_inff();
                top = fmaxf(top, all[i]);
            }
        }
        top = wave_max(top);
#pragma unroll
        for (int i = 0; i < kMax; ++i) {
            w[i] = id[i] >= 0 ? expf(l[i] - top) : 0.f;
            if (kRenorm) sum += w[i];
        }
        if constexpr (!kRenorm) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                all[i] = 4 * lane + i < E ? expf(all[i] - top) : 0.f;
                sum += all[i];
            }
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int i = 0; i < kMax; ++i) dot += w[i] / sum * dw[i];
        dot = wave_sum(dot);
#pragma unroll
        for (int i = 0; i < kMax; ++i) d[i] = kRenorm ? w[i] / sum * (dw[i] - dot) : w[i] / sum * dw[i];
        if constexpr (!kRenorm) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = -all[i] / sum * dot;
        }
    }
    for (int j = 0; j < k; ++j) {  // each pick to its expert's lane
        int e = 0;
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kMax; ++i)
            if (j >> 6 == i) {
                e = __shfl(id[i], j & 63);
                v = __shfl(d[i], j & 63);
            }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e == 4 * lane + i) acc[i] += v;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (4 * lane + i < E) store1(dlogits + t * E + 4 * lane + i, acc[i]);
}

// Between what lanes of a wave write to LDS for one another and what these read of it: the wave's LDS accesses run in
// their order, so this costs no wait, but each lane's own program does not show the compiler that they meet.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The same for at most eight picks where nothing runs over all E: a wave takes eight tokens, a pick in each lane, and
// puts their rows together in LDS. 16384 tokens of 256 experts take 5.6 us in a graph (5.3 with 1 - s taken from s, where a
// wave for each token took 11.1).
template <int kCtrl>
__device__ __forceinline__ float lane_swap(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, 0xf, 0xf, false));
}
template <typename F>
__device__ __forceinline__ float over_eight(float v, F f) {  // over eight neighbouring lanes, the same in each
    v = f(v, lane_swap<0xb1>(v));   // lane ^ 1
    v = f(v, lane_swap<0x4e>(v));   // lane ^ 2
    return f(v, lane_swap<0x141>(v));  // half mirror: lane ^ 7, of the other four
}

template <typename TO, bool kSigmoid, bool kRenorm>
__global__ __launch_bounds__(256) void route_grad_few_kernel(const float* __restrict__ logits,
                                                             const int32_t* __restrict__ ids,
                                                             const float* __restrict__ dtopk_w, int T, int E, int k,
                                                             bool vec, TO* __restrict__ dlogits) {
    __shared__ __attribute__((aligned(16))) float rows[4][8 * kGateMaxE];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane & 7;
    float* row = rows[wave];
    const long t0 = ((long)blockIdx.x * 4 + wave) * 8, t = t0 + (lane >> 3);
    const bool pick = t < T && j < k;
    int id = pick ? ids[t * k + j] : -1;
    float dw = pick ? dtopk_w[t * k + j] : 0.f;
    if ((unsigned)id >= (unsigned)E) id = -1;
    const float l = id >= 0 ? logits[t * E + id] : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<f32x4*>(row + i * kGateMaxE + 4 * lane) = f32x4{0.f, 0.f, 0.f, 0.f};
    auto add = [](float a, float b) { return a + b; };
    auto most = [](float a, float b) { return fmaxf(a, b); };
    if (id < 0) dw = 0.f;
    float d;
    if constexpr (kSigmoid) {
        const Sigmoid sig = sigmoid_of(l);
        const float s = id >= 0 ? sig.s : 0.f;
        if constexpr (kRenorm) {
            const float w = s / over_eight(s, add), dot = over_eight(w * dw, add);
            d = w * sig.rest * (dw - dot);
        } else {
            d = s * sig.rest * dw;
        }
    } else {
        const float top = over_eight(id >= 0 ? l : -__builtin_inff(), most);
        const float e = id >= 0 ? expf(l - top) : 0.f;
        const float w = e / over_eight(e, add), dot = over_eight(w * dw, add);
        d = w * (dw - dot);
    }
    // one pick of each token at a time, in order: an id that stands twice gets both
    wave_sync();
    for (int i = 0; i < k; ++i) {
        if (j == i && id >= 0) row[(lane >> 3) * kGateMaxE + id] += d;
        wave_sync();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (t0 + i >= T) break;
        const f32x4 v = *reinterpret_cast<const f32x4*>(row + i * kGateMaxE + 4 * lane);
        TO* o = dlogits + (t0 + i) * E + 4 * lane;
        if (vec) {
            if (4 * lane < E) {
                if constexpr (sizeof(TO) == 2)
                    *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                else *reinterpret_cast<f32x4*>(o) = v;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (4 * lane + e < E) store1(o + e, v[e]);
        }
    }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

Dropout dropout_of(float p, const void* rng) {
    const uint32_t t = dropout_threshold(p);
    return Dropout{(const uint64_t*)rng, t, 65536.0f / (float)(65536u - t)};
}

// tokens of one launch, at most: a grid of 2^32 work items and more runs short without an error
constexpr int kTokens = 1 << 21;

int blocks_for(long threads) {
    return (int)std::max(1L, std::min((threads + 255) / 256, (long)device_info().cu_count * 16));
}

}  // namespace

moe_status launch_dropout(const void* x, const void* residual, moe_dtype dt, long n, float p, const void* rng,
                          void* out, hipStream_t st) {
    const bool vec = aligned16(x) && aligned16(residual) && aligned16(out);
    const Dropout d = dropout_of(p, rng);
#define DROP(T, VEC)                                                                                             \
    hipLaunchKernelGGL((dropout_kernel<T, VEC>), dim3(blocks_for((n + 7) / 8)), dim3(256), 0, st, (const T*)x, \
                       (const T*)residual, n, d, (T*)out)
    if (dt == MOE_BF16 && vec) DROP(uint16_t, true);
    else if (dt == MOE_BF16) DROP(uint16_t, false);
    else if (vec) DROP(float, true);
    else DROP(float, false);
#undef DROP
    return check_launch("dropout_kernel");
}

moe_status launch_swiglu(const void* gu, const void* da, moe_dtype dt, const int32_t* n_rows, int max_rows, int I,
                         float p, const void* rng, void* dgu, void* a, hipStream_t st) {
    const bool vec = I % 8 == 0 && aligned16(gu) && aligned16(da) && aligned16(dgu) && aligned16(a);
    const Dropout d = dropout_of(p, rng);
    const dim3 grid(blocks_for((long)max_rows * ((I + 7) / 8)));
#define UNITS(T, VEC, GRAD)                                                                                       \
    hipLaunchKernelGGL((swiglu_kernel<T, VEC, GRAD>), grid, dim3(256), 0, st, (const T*)gu, (const T*)da, n_rows, \
                       max_rows, I, d, (T*)dgu, (T*)a)
#define UNITS_OF(T)                 \
    if (vec && da) UNITS(T, true, true);  \
    else if (vec) UNITS(T, true, false);  \
    else if (da) UNITS(T, false, true);   \
    else UNITS(T, false, false)
    if (dt == MOE_BF16) {
        UNITS_OF(uint16_t);
    } else {
        UNITS_OF(float);
    }
#undef UNITS_OF
#undef UNITS
    return check_launch("swiglu_kernel");
}

moe_status launch_combine_grad(const void* dout, const void* y, moe_dtype dt, const int32_t* slot_to_row,
                               const float* topk_w, int T, int k, int H, const int32_t* offsets, int shared_group,
                               void* dy, float* dw, hipStream_t st) {
    const bool vec = H % 8 == 0 && aligned16(dout) && aligned16(y) && aligned16(dy);
    const int most = kTokens / ((k + kPicks - 1) / kPicks);
    for (int t0 = 0; t0 < T;) {
        const int n = std::min(T - t0, most);
        // picks are spread over workgroups until there are about four of these per CU
        const int per = std::max(1, (int)std::min((long)std::min(k, kPicks), (long)n * k / 1024));
        const CombineGrad p{dout, y, slot_to_row, topk_w, t0, T, k, H, offsets, shared_group, per, dy, dw};
        const dim3 grid(n, (k + per - 1) / per);
#define CGRAD(T, VEC, CHUNKS) hipLaunchKernelGGL((combine_grad_kernel<T, VEC, CHUNKS>), grid, dim3(256), 0, st, p)
#define CGRAD_OF(T, VEC)                  \
    if (H <= 2048) CGRAD(T, VEC, 1);      \
    else if (H <= 4096) CGRAD(T, VEC, 2); \
    else if (H <= 8192) CGRAD(T, VEC, 4); \
    else CGRAD(T, VEC, 0)
        if (dt == MOE_BF16 && vec) {
            CGRAD_OF(uint16_t, true);
        } else if (dt == MOE_BF16) {
            CGRAD_OF(uint16_t, false);
        } else if (vec) {
            CGRAD_OF(float, true);
        } else {
            CGRAD_OF(float, false);
        }
#undef CGRAD_OF
#undef CGRAD
        t0 += n;
    }
    return check_launch("combine_grad_kernel");
}

moe_status launch_route_grad(const float* logits, const int32_t* ids, const float* dtopk_w, int T, int E, int k,
                             int scoring, int renorm, void* dlogits, moe_dtype out_dt, hipStream_t st) {
    for (; T > kTokens; T -= kTokens) {
        const moe_status s = launch_route_grad(logits, ids, dtopk_w, kTokens, E, k, scoring, renorm, dlogits, out_dt, st);
        if (s != MOE_OK) return s;
        logits += (size_t)kTokens * E;
        ids += (size_t)kTokens * k;
        dtopk_w += (size_t)kTokens * k;
        dlogits = (uint8_t*)dlogits + (size_t)kTokens * E * (out_dt == MOE_BF16 ? 2 : 4);
    }
    if (k <= 8 && (scoring == MOE_SIGMOID || renorm)) {
        const dim3 few((T + 31) / 32);
        const bool vec = E % 4 == 0 && aligned16(dlogits);
#define GATE(TO, SIG, REN)                                                                                           \
    hipLaunchKernelGGL((route_grad_few_kernel<TO, SIG, REN>), few, dim3(256), 0, st, logits, ids, dtopk_w, T, E, k, \
                       vec, (TO*)dlogits)
#define GATE_OF(TO)                                              \
    if (scoring == MOE_SIGMOID && renorm) GATE(TO, true, true);  \
    else if (scoring == MOE_SIGMOID) GATE(TO, true, false);      \
    else GATE(TO, false, true)
        if (out_dt == MOE_BF16) {
            GATE_OF(uint16_t);
        } else {
            GATE_OF(float);
        }
#undef GATE_OF
#undef GATE
        return check_launch("route_grad_few_kernel");
    }
    const dim3 grid((T + 3) / 4);
#define GATE(TO, SIG, REN)                                                                                           \
    hipLaunchKernelGGL((route_grad_kernel<TO, SIG, REN>), grid, dim3(256), 0, st, logits, ids, dtopk_w, T, E, k, \
                       (TO*)dlogits)
#define GATE_OF(TO)                                         \
    if (scoring == MOE_SIGMOID && renorm) GATE(TO, true, true);  \
    else if (scoring == MOE_SIGMOID) GATE(TO, true, false);      \
    else if (renorm) GATE(TO, false, true);                      \
    else GATE(TO, false, false)
    if (out_dt == MOE_BF16) {
        GATE_OF(uint16_t);
    } else {
        GATE_OF(float);
    }
#undef GATE_OF
#undef GATE
    return check_launch("route_grad_kernel");
}

}  // namespace moe
