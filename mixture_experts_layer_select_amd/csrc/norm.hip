// The norms around the MoE block with its residual: the residual add and RMS
// norm before it, and the routing-weighted combine, post norm, gate, residual
// scale and residual behind it, each in one pass over its rows.
//
// One workgroup per token keeps the token's row in registers (one or two chunks
// of 8 columns a thread), so each input is read once: the sum of squares is
// taken while the row is held. Bound by HBM for many tokens, by memory latency
// for a few. Sums are fp32 in a fixed order. At H = 7168 in bf16: 16383 rows of
// the norm 162 us (5.8 TB/s), 4097 tokens of eight picks and a shared row 134 us
// (5.0 TB/s), one row 4 us, 16 tokens 5.7 us.
#include "combine_dev.h"

namespace moe {
namespace {

constexpr int kNormMaxH = 16384;
// rows of one launch, at most: a grid of 2^32 work items and more (2^26 rows of one wave) runs short without an error
constexpr int kNormRows = 1 << 21;

// sum over the workgroup, the same in every thread
template <int kThreads>
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) v += __shfl_xor(v, s);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) t += red[i];
    return t;
}

// A row's bytes at the element's own alignment: the hardware takes vector
// accesses there too, only slower where they cross a line. 16000 rows of 7171
// bf16 columns take 200 us so, and 626 element by element.
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Eight {
    T e[8];
};

// eight columns from h (kVec: one aligned vector or two; otherwise at the
// element's alignment, and element by element where H ends, zeros past it)
template <bool kVec, typename T>
__device__ __forceinline__ void get8(const T* p, int h, int H, float* v) {
    if constexpr (kVec) {
        load8(p + h, v);
    } else if (h + 8 <= H) {
        alignas(16) Eight<T> t = *reinterpret_cast<const Eight<T>*>(p + h);
        load8(t.e, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = load1(p + min(h + i, H - 1));  // no branches: the loads overlap
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = h + i < H ? v[i] : 0.f;
    }
}
template <bool kVec, typename T>
__device__ __forceinline__ void put8(T* p, int h, int H, const float* v) {
    if constexpr (kVec) {
        store8(p + h, v);
    } else if (h + 8 <= H) {
        alignas(16) Eight<T> t;
        store8(t.e, v);
        *reinterpret_cast<Eight<T>*>(p + h) = t;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (h + i < H) store1(p + h + i, v[i]);
    }
}

// h_out may be x or delta: neither they nor the outputs are __restrict__. A thread has loaded all its columns of a row
// before it stores the first.
template <typename T, bool kVec, int kThreads, int kChunks>
__global__ __launch_bounds__(kThreads) void pre_norm_kernel(const T* x, const T* delta, float scale,
                                                            const float* __restrict__ gain, float eps, int t0, int H,
                                                            T* h_out, T* n_out) {
    __shared__ float red[kThreads / 64];
    const size_t row = (size_t)(t0 + (int)blockIdx.x) * H;
    float v[kChunks][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int h = (c * kThreads + threadIdx.x) * 8;
        if (h < H) get8<kVec>(x + row, h, H, v[c]);
    }
    if (delta) {
        float d[kChunks][8];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int h = (c * kThreads + threadIdx.x) * 8;
            if (h < H) get8<kVec>(delta + row, h, H, d[c]);
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] = __builtin_fmaf(scale, d[c][i], v[c][i]);
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int h = (c * kThreads + threadIdx.x) * 8;
        if (h < H) {
            if (h_out) put8<kVec>(h_out + row, h, H, v[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(v[c][i], v[c][i], ss);
        }
    }
    const float r = 1.0f / sqrtf(block_sum<kThreads>(ss, red) / (float)H + eps);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int h = (c * kThreads + threadIdx.x) * 8;
        if (h < H) {
            float g[8];
            if (gain) get8<kVec>(gain, h, H, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] = gain ? v[c][i] * r * g[i] : v[c][i] * r;
            put8<kVec>(n_out + row, h, H, v[c]);
        }
    }
}

struct CombineNorm {
    int t0;  // first token of the launch
    const void* y;
    const int32_t* slot_to_row;
    const float* topk_w;
    int T, k, H;
    const int32_t* offsets;
    int shared_group;
    const float* gain;  // null: no norm
    float eps;
    const void* gate;   // null: 1
    int gate_rows;
    float alpha;
    const void* residual;  // null: 0
    void* out;
};

template <typename TY, typename TO, bool kVec, int kThreads, int kChunks>
__global__ __launch_bounds__(kThreads) void combine_norm_kernel(CombineNorm p) {
    __shared__ float red[kThreads / 64];
    const int t = p.t0 + (int)blockIdx.x, H = p.H;
    const TY* y = (const TY*)p.y;
    float acc[kChunks][8] = {};
    auto add = [&](int row, float w) {
        const TY* yr = y + (size_t)row * H;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int h = (c * kThreads + threadIdx.x) * 8;
            if (h < H) {
                float v[8];
                get8<kVec>(yr, h, H, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[c][i] = __builtin_fmaf(w, v[i], acc[c][i]);
            }
        }
    };
    for (int j = 0; j < p.k; ++j) {
        const int row = p.slot_to_row[(size_t)t * p.k + j];
        if (row >= 0) add(row, p.topk_w[(size_t)t * p.k + j]);
    }
    if (p.shared_group >= 0) add(p.offsets[p.shared_group] + t, 1.0f);
    float r = 1.0f;
    if (p.gain) {
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(acc[c][i], acc[c][i], ss);
        r = 1.0f / sqrtf(block_sum<kThreads>(ss, red) / (float)H + p.eps);
    }
    const TO* gate = (const TO*)p.gate + (p.gate_rows > 1 ? (size_t)t * H : 0);
    const TO* res = (const TO*)p.residual + (size_t)t * H;
    TO* out = (TO*)p.out + (size_t)t * H;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int h = (c * kThreads + threadIdx.x) * 8;
        if (h < H) {
            float v[8], g[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = acc[c][i] * r;
            if (p.gain) {
                get8<kVec>(p.gain, h, H, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= g[i];
            }
            if (p.gate) {
                get8<kVec>(gate, h, H, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= g[i];
            }
            float s[8] = {};
            if (p.residual) get8<kVec>(res, h, H, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = __builtin_fmaf(p.alpha, v[i], s[i]);
            put8<kVec>(out, h, H, s);
        }
    }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Threads by the row's width, so that nearly all of them hold columns: rows of
// 512 columns take 12 us per 16000 with one wave each and 17 with four, rows of
// 4096 44 us per 8000 with 512 threads and 55 with 1024, rows of 7168 163 us
// per 16000 with 512 threads of two chunks each and 164 with 1024 of one. The
// combine, whose picks' rows follow one another, has those on 1024: 134 us for
// 4097 tokens, 137 on 512.
template <typename T, bool kVec>
void pre_norm_sized(const void* x, const void* delta, float scale, const float* gain, float eps, int T_, int H,
                    void* h_out, void* n_out, hipStream_t st) {
    for (int t0 = 0; t0 < T_;) {
        const dim3 grid(std::min(T_ - t0, kNormRows));
#define PRE(THREADS, CHUNKS)                                                                                 \
    hipLaunchKernelGGL((pre_norm_kernel<T, kVec, THREADS, CHUNKS>), grid, dim3(THREADS), 0, st, (const T*)x, \
                       (const T*)delta, scale, gain, eps, t0, H, (T*)h_out, (T*)n_out)
        if (H <= 512) PRE(64, 1);
        else if (H <= 2048) PRE(256, 1);
        else if (H <= 4096) PRE(512, 1);
        else if (H <= 8192) PRE(512, 2);
        else PRE(1024, 2);
#undef PRE
        t0 += (int)grid.x;
    }
}

template <typename TY, typename TO, bool kVec>
void combine_norm_sized(CombineNorm p, hipStream_t st) {
    while (p.t0 < p.T) {
        const dim3 grid(std::min(p.T - p.t0, kNormRows));
#define POST(THREADS, CHUNKS) \
    hipLaunchKernelGGL((combine_norm_kernel<TY, TO, kVec, THREADS, CHUNKS>), grid, dim3(THREADS), 0, st, p)
        if (p.H <= 512) POST(64, 1);
        else if (p.H <= 2048) POST(256, 1);
        else if (p.H <= 4096) POST(512, 1);
        else if (p.H <= 8192) POST(1024, 1);
        else POST(1024, 2);
#undef POST
        p.t0 += (int)grid.x;
    }
}

template <typename TY, typename TO>
void combine_norm_typed(const CombineNorm& p, hipStream_t st) {
    const bool vec = p.H % 8 == 0 && aligned16(p.y) && aligned16(p.gain) && aligned16(p.gate) &&
                     aligned16(p.residual) && aligned16(p.out);
    if (vec) combine_norm_sized<TY, TO, true>(p, st);
    else combine_norm_sized<TY, TO, false>(p, st);
}

}  // namespace

bool norm_h_supported(int H) { return H <= kNormMaxH; }

moe_status launch_pre_norm(const void* x, const void* delta, float delta_scale, const float* gain, float eps,
                           moe_dtype dt, int T, int H, void* h_out, void* n_out, hipStream_t st) {
    const bool vec = H % 8 == 0 && aligned16(x) && aligned16(delta) && aligned16(gain) && aligned16(h_out) &&
                     aligned16(n_out);
    if (dt == MOE_BF16 && vec)
        pre_norm_sized<uint16_t, true>(x, delta, delta_scale, gain, eps, T, H, h_out, n_out, st);
    else if (dt == MOE_BF16)
        pre_norm_sized<uint16_t, false>(x, delta, delta_scale, gain, eps, T, H, h_out, n_out, st);
    else if (vec)
        pre_norm_sized<float, true>(x, delta, delta_scale, gain, eps, T, H, h_out, n_out, st);
    else
        pre_norm_sized<float, false>(x, delta, delta_scale, gain, eps, T, H, h_out, n_out, st);
    return check_launch("pre_norm_kernel");
}

moe_status launch_combine_norm(const void* y_perm, moe_dtype y_dt, const int32_t* slot_to_row,
                               const float* topk_w, int T, int k, int H, const int32_t* offsets,
                               int shared_group, const float* gain, float eps, const void* gate, int gate_rows,
                               float alpha, const void* residual, void* out, moe_dtype out_dt, hipStream_t st) {
    const CombineNorm p{0, y_perm, slot_to_row, topk_w, T, k, H, offsets, shared_group, gain, eps, gate, gate_rows,
                        alpha, residual, out};
    if (y_dt == MOE_BF16 && out_dt == MOE_BF16) combine_norm_typed<uint16_t, uint16_t>(p, st);
    else if (y_dt == MOE_BF16) combine_norm_typed<uint16_t, float>(p, st);
    else if (out_dt == MOE_BF16) combine_norm_typed<float, uint16_t>(p, st);
    else combine_norm_typed<float, float>(p, st);
    return check_launch("combine_norm_kernel");
}

}  // namespace moe
