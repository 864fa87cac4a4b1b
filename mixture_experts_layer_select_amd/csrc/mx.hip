// Experts in microscaled 4-bit floating point (OCP MXFP4, mx_dev.h): the
// quantisation of rows, its inverse, and the grouped expert GEMMs with both
// operands in that format.
#include "ffn_dev.h"
#include "mx_dev.h"

namespace moe {
namespace {

// ============================================================================ quantisation
// Rows are whole blocks of 32, so a tensor is a flat list of blocks: four
// lanes hold a block, eight values each, and agree on its largest by two DPP
// moves. Bound by HBM.
template <typename TIn>
__device__ __forceinline__ void load_eight(const TIn* p, float* v);
template <>
__device__ __forceinline__ void load_eight<uint16_t>(const uint16_t* p, float* v) {
    const u32x4 q = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(q[i]);
        v[2 * i + 1] = bf16_hi(q[i]);
    }
}
template <>
__device__ __forceinline__ void load_eight<float>(const float* p, float* v) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
    }
}

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_max_u32(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xf, 0xf, false);
    return o > v ? o : v;
}

template <typename TIn>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const TIn* __restrict__ x, long n_eight,
                                                          uint32_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n_eight; i += (long)gridDim.x * 256) {
        float v[8];
        load_eight<TIn>(x + i * 8, v);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
        m = dpp_max_u32<0xb1>(m);  // lane ^ 1; n_eight is a multiple of 4, so the four lanes run together
        m = dpp_max_u32<0x4e>(m);  // lane ^ 2
        const uint32_t byte = mx_scale_byte(m);
        codes[i] = mx_pack8(v, mx_inverse(byte));
        if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
    }
}

// E2M1 code (4 bits) -> fp32
__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t m = c & 7u;
    // 0, 0.5, then 1.m * 2^(exp - 1)
    const float v = m < 2 ? 0.5f * (float)m : __uint_as_float((126u + (m >> 1)) << 23 | (m & 1u) << 22);
    return (c & 8u) ? -v : v;
}

template <typename TOut>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, long n_eight,
                                                            TOut* __restrict__ out) {
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n_eight; i += (long)gridDim.x * 256) {
        const uint32_t c = codes[i], byte = scales[i >> 2];
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = __builtin_ldexpf(e2m1_value(c >> (4 * j) & 15u), (int)byte - 127);
            if (byte == kMxNan) v[j] = __uint_as_float(0x7fc00000u);
        }
        if constexpr (sizeof(TOut) == 2) {  // two significant bits: exact in bf16, denormals included
            *reinterpret_cast<u32x4*>(out + i * 8) =
                u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
        } else {
            *reinterpret_cast<f32x4*>(out + i * 8) = f32x4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4*>(out + i * 8 + 4) = f32x4{v[4], v[5], v[6], v[7]};
        }
    }
}

// ============================================================================ grouped GEMMs
// Items are (m-tile of at most 64 rows, n-block of 128 weight rows); wave w
// owns weight rows 32w + [0, 32) (SwiGLU: 16 gate and 16 up rows in the two
// halves of its MFMA rows) and both 32-row halves of the tile. Fragments come
// straight from global memory.
constexpr int kMxTM = 64;

// weight row (within the wave's 32) that MFMA row rho reads: lane (l31, hi)
// then holds the D values of 16 consecutive weight rows 16 hi + [0, 16)
__device__ __forceinline__ int mx_row_of(int rho) { return 16 * ((rho >> 2) & 1) + 4 * (rho >> 3) + (rho & 3); }

struct MxGemm {
    const uint8_t* x;         // activation codes, rows of K/2 bytes
    const uint8_t* xs;        // their scales, rows of K/32 bytes
    const uint8_t *w, *ws, *wsh, *wsh_s;  // routed and shared weights and scales
    const int32_t* offsets;
    int n_routed, n_groups, max_rows, K, Nw, NB;
    uint8_t* out;             // SwiGLU: A codes [max_rows][I/2]; down: y [max_rows][H] bf16
    uint8_t* out_scale;       // SwiGLU: [max_rows][I/32]
    ActSrc src;
};

template <bool kSwiGLU, bool kGather>
__global__ __launch_bounds__(256) void mx_gemm_kernel(MxGemm p) {
    __shared__ TileMap tm;
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int l31 = lane & 31, hi = lane >> 5;
    const int K = p.K, kb = K / kMxBlock;
    const int n_items = build_tile_map(tm, p.offsets, p.n_groups, p.max_rows, kMxTM) * p.NB;
    const int I = p.Nw / 2;  // SwiGLU: intermediate size
    for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
        int nb;
        const MTile tile = item_at(tm, p.offsets, p.n_groups, p.max_rows, item, p.NB, kMxTM, nb);
        const bool routed = tile.group < p.n_routed;
        const uint8_t* W = routed ? p.w + (size_t)tile.group * p.Nw * (K / 2) : p.wsh;
        const uint8_t* Ws = routed ? p.ws + (size_t)tile.group * p.Nw * kb : p.wsh_s;
        // SwiGLU: the wave's 32 intermediate columns, gate rows then up rows
        constexpr int kSets = kSwiGLU ? 2 : 1;
        const int n0 = nb * 128 + 32 * wave;
        const uint8_t *wr[kSets], *sr[kSets];
#pragma unroll
        for (int s = 0; s < kSets; ++s) {
            const size_t row = (size_t)s * I + n0 + mx_row_of(l31);
            wr[s] = W + row * (K / 2) + 16 * hi;
            sr[s] = Ws + row * kb + hi;
        }
        const uint8_t *xr[2], *xsr[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = min(32 * j + l31, tile.rows - 1);
            long row = tile.row0 + r;
            if (kGather) {
                const int slot = p.src.row_slot[row];
                row = slot < p.src.S ? slot / p.src.k : slot - p.src.S;
                row = max(0L, min(row, (long)p.src.rows - 1));
            }
            xr[j] = p.x + (size_t)row * (K / 2) + 16 * hi;
            xsr[j] = p.xs + (size_t)row * kb + hi;
        }
        f32x16 acc[kSets][2] = {};
        for (int c = 0; c < K / 64; ++c) {
            u32x4 b[2];
            uint32_t sb[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                b[j] = *reinterpret_cast<const u32x4*>(xr[j] + 32 * c);
                sb[j] = xsr[j][2 * c];
            }
#pragma unroll
            for (int s = 0; s < kSets; ++s) {
                const u32x4 a = *reinterpret_cast<const u32x4*>(wr[s] + 32 * c);
                const uint32_t sa = sr[s][2 * c];
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[s][j] = mfma_fp4<0, 0>(a, b[j], acc[s][j], sa, sb[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int m = 32 * j + l31;
            const size_t row = (size_t)tile.row0 + m;
            if constexpr (kSwiGLU) {
                float v[16];
                uint32_t mx = 0;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    v[r] = silu_mul(acc[0][j][r], acc[1][j][r]);
                    mx = max(mx, abs_bits(v[r]));
                }
                mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32));
                const uint32_t byte = mx_scale_byte(mx);
                const float inv = mx_inverse(byte);
                if (m < tile.rows) {
                    *reinterpret_cast<uint2*>(p.out + row * (I / 2) + n0 / 2 + 8 * hi) =
                        make_uint2(mx_pack8(v, inv), mx_pack8(v + 8, inv));
                    if (hi == 0) p.out_scale[row * (I / kMxBlock) + n0 / kMxBlock] = (uint8_t)byte;
                }
            } else if (m < tile.rows) {
                uint16_t* y = reinterpret_cast<uint16_t*>(p.out) + row * p.Nw + n0 + 16 * hi;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const f32x16& a = acc[0][j];
                    *reinterpret_cast<u32x4*>(y + 8 * q) =
                        u32x4{pack_bf16x2(a[8 * q], a[8 * q + 1]), pack_bf16x2(a[8 * q + 2], a[8 * q + 3]),
                              pack_bf16x2(a[8 * q + 4], a[8 * q + 5]), pack_bf16x2(a[8 * q + 6], a[8 * q + 7])};
                }
            }
        }
    }
}

// workspace: A codes [max_rows][I/2] | A scales [max_rows][I/32]
size_t mx_scale_offset(const moe_expert_weights* w, int max_rows) {
    return align_up((size_t)max_rows * (w->I / 2), 256);
}

template <bool kSwiGLU, bool kGather>
moe_status launch_gemm(const MxGemm& p, hipStream_t st) {
    const long tiles = (long)(p.max_rows + kMxTM - 1) / kMxTM + p.n_groups;
    const int grid = (int)std::min(tiles * p.NB, (long)device_info().cu_count * 2);
    hipLaunchKernelGGL((mx_gemm_kernel<kSwiGLU, kGather>), dim3(grid), dim3(256), 0, st, p);
    return check_launch("mx_gemm_kernel");
}

}  // namespace

moe_status launch_mx_quantize(const void* x, moe_dtype x_dt, long rows, int cols, void* codes, void* scales,
                              hipStream_t st) {
    const long n = rows * (cols / 8);
    const int blocks = (int)std::min((n + 255) / 256, (long)device_info().cu_count * 16);
    if (x_dt == MOE_BF16)
        hipLaunchKernelGGL(mx_quantize_kernel<uint16_t>, dim3(blocks), dim3(256), 0, st, (const uint16_t*)x, n,
                           (uint32_t*)codes, (uint8_t*)scales);
    else
        hipLaunchKernelGGL(mx_quantize_kernel<float>, dim3(blocks), dim3(256), 0, st, (const float*)x, n,
                           (uint32_t*)codes, (uint8_t*)scales);
    return check_launch("mx_quantize_kernel");
}

moe_status launch_mx_dequantize(const void* codes, const void* scales, long rows, int cols, void* out,
                                moe_dtype out_dt, hipStream_t st) {
    const long n = rows * (cols / 8);
    const int blocks = (int)std::min((n + 255) / 256, (long)device_info().cu_count * 16);
    if (out_dt == MOE_BF16)
        hipLaunchKernelGGL(mx_dequantize_kernel<uint16_t>, dim3(blocks), dim3(256), 0, st, (const uint32_t*)codes,
                           (const uint8_t*)scales, n, (uint16_t*)out);
    else
        hipLaunchKernelGGL(mx_dequantize_kernel<float>, dim3(blocks), dim3(256), 0, st, (const uint32_t*)codes,
                           (const uint8_t*)scales, n, (float*)out);
    return check_launch("mx_dequantize_kernel");
}

size_t mx_ffn_workspace_bytes(const moe_expert_weights* w, int max_rows) {
    return mx_scale_offset(w, max_rows) + align_up((size_t)max_rows * (w->I / kMxBlock), 256) + 256;
}

moe_status launch_mx_gate_up(const moe_expert_weights* w, const void* x, const void* x_scale,
                             const int32_t* offsets, int n_groups, int max_rows, void* ws, hipStream_t st,
                             const ActSrc& src) {
    MxGemm p{};
    p.x = (const uint8_t*)x;
    p.xs = (const uint8_t*)x_scale;
    p.w = (const uint8_t*)w->w13;
    p.ws = (const uint8_t*)w->w13_scale;
    p.wsh = (const uint8_t*)w->ws13;
    p.wsh_s = (const uint8_t*)w->ws13_scale;
    p.offsets = offsets;
    p.n_routed = w->E_local;
    p.n_groups = n_groups;
    p.max_rows = max_rows;
    p.K = w->H;
    p.Nw = 2 * w->I;
    p.NB = w->I / 128;
    p.out = (uint8_t*)ws;
    p.out_scale = (uint8_t*)ws + mx_scale_offset(w, max_rows);
    p.src = src;
    return src.row_slot ? launch_gemm<true, true>(p, st) : launch_gemm<true, false>(p, st);
}

moe_status launch_mx_down(const moe_expert_weights* w, const int32_t* offsets, int n_groups, int max_rows,
                          void* y_perm, void* ws, hipStream_t st) {
    MxGemm p{};
    p.x = (const uint8_t*)ws;
    p.xs = (const uint8_t*)ws + mx_scale_offset(w, max_rows);
    p.w = (const uint8_t*)w->w2;
    p.ws = (const uint8_t*)w->w2_scale;
    p.wsh = (const uint8_t*)w->ws2;
    p.wsh_s = (const uint8_t*)w->ws2_scale;
    p.offsets = offsets;
    p.n_routed = w->E_local;
    p.n_groups = n_groups;
    p.max_rows = max_rows;
    p.K = w->I;
    p.Nw = w->H;
    p.NB = w->H / 128;
    p.out = (uint8_t*)y_perm;
    return launch_gemm<false, false>(p, st);
}

}  // namespace moe
