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
// Items are (m-tile of at most 256 rows, n-block of 256 weight rows); one
// workgroup of 4 waves per CU walks them (item_at's order, a contiguous slice
// per XCD). Both operands of each K step of 128 arrive in a 4-stage LDS ring
// by direct global->LDS loads, three steps ahead; the E8M0 scales of four
// steps come in one 16-byte piece per row and sit in registers for them.
//
// Waves form a 2 x 2 grid: wave (wm, wn) owns the 32-token blocks 2j + wm of
// the tile and 128 weight rows, as 4 x NX blocks of 32x32 accumulators, NX =
// 1, 2 or 4 by the tile's height (64, 128, 256 rows): a short tile loads only
// its own rows, so a group of up to 256 rows reads its weights from HBM once
// and little else.
//   SwiGLU: LDS rows q < 128 are gate rows nb*128 + q, q >= 128 the up rows I +
//     nb*128 + q - 128; wave wn owns gate q = 64wn + [0, 64) (s = 0, 1) and
//     the up rows 128 + the same (s = 2, 3).
//   Down: q -> w2 row nb*256 + q; wave wn owns q = 128wn + 32s + [0, 32).
// LDS rows are 64 bytes; chunk c of row q sits at chunk c ^ mx_swz(q), which
// spreads the 16 rows that a quarter of a wave reads over all 64 banks.
constexpr int kMxTM = 256;     // tokens per tile
constexpr int kMxTN = 256;     // weight rows per tile
constexpr int kMxThreads = 256;
constexpr int kMxStepB = 64;   // bytes of a row per K step of 128
constexpr int kMxPanel = 4;    // m-tiles per item panel

struct MxStage {
    uint8_t w[kMxTN * kMxStepB];  // 16 KB
    uint8_t x[kMxTM * kMxStepB];  // 16 KB
};
struct MxScales {  // four K steps
    uint8_t w[kMxTN * 16];
    uint8_t x[kMxTM * 16];
};

// weight row (within the wave's 32) that MFMA row rho reads: lane (l31, hi)
// then holds the D values of 16 consecutive weight rows 16 hi + [0, 16), so
// it writes 16 neighbouring outputs
__device__ __forceinline__ int mx_row_of(int rho) { return 16 * ((rho >> 2) & 1) + 4 * (rho >> 3) + (rho & 3); }
// chunk swizzles: weight rows are read in mx_row_of's order, tokens in rows'
__device__ __forceinline__ int mx_swz_w(int q) { return (((q >> 2) ^ (q >> 1)) & 1) | ((q >> 4) & 1) << 1; }
__device__ __forceinline__ int mx_swz_x(int q) { return (((q >> 1) ^ (q >> 3)) & 1) | ((q >> 2) & 1) << 1; }

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
__global__ __launch_bounds__(kMxThreads, 1) void mx_gemm_kernel(MxGemm p) {
    // one object per stage: the compiler tells the one being filled from the one being read
    __shared__ __attribute__((aligned(1024))) MxStage st0;
    __shared__ __attribute__((aligned(1024))) MxStage st1;
    __shared__ __attribute__((aligned(1024))) MxStage st2;
    __shared__ __attribute__((aligned(1024))) MxStage st3;
    __shared__ __attribute__((aligned(1024))) MxScales sc;
    __shared__ TileMap tm;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int l31 = lane & 31, hi = lane >> 5;
    const int K = p.K, kb = K / kMxBlock, rowb = K / 2;
    const int nk = K / 128;
    const int I = p.Nw / 2;  // SwiGLU: intermediate size
    const int n_items = build_tile_map(tm, p.offsets, p.n_groups, p.max_rows, kMxTM) * p.NB;
    const int xcd = blockIdx.x & 7;
    const int per_xcd = gridDim.x >> 3;
    const int i_lo = (int)((long)n_items * xcd / 8);
    const int i_hi = (int)((long)n_items * (xcd + 1) / 8);

    // fragment offsets in a stage: weight tile s at off + q0(s) * 64, token block j at off + j * 4096
    const int rw = mx_row_of(l31);
    int offa[2], offb[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        offa[h] = rw * kMxStepB + ((2 * h + hi) ^ mx_swz_w(rw)) * 16;
        offb[h] = (32 * wm + l31) * kMxStepB + ((2 * h + hi) ^ mx_swz_x(l31)) * 16;
    }
    auto q0 = [&](int s) { return kSwiGLU ? 128 * (s >> 1) + 64 * wn + 32 * (s & 1) : 128 * wn + 32 * s; };

    for (int item = i_lo + (int)(blockIdx.x >> 3); item < i_hi; item += per_xcd) {
        int nb_v;
        const MTile tile_v = item_at(tm, p.offsets, p.n_groups, p.max_rows, item, p.NB, kMxTM, nb_v, kMxPanel);
        const int nb = __builtin_amdgcn_readfirstlane(nb_v);
        const MTile tile{__builtin_amdgcn_readfirstlane(tile_v.group), __builtin_amdgcn_readfirstlane(tile_v.row0),
                         __builtin_amdgcn_readfirstlane(tile_v.rows)};
        const bool routed = tile.group < p.n_routed;
        const __amdgpu_buffer_rsrc_t w_d = buffer_rsrc(
            routed ? p.w + (size_t)tile.group * p.Nw * rowb : p.wsh, clamp_bytes((size_t)p.Nw * rowb));
        const __amdgpu_buffer_rsrc_t ws_d =
            buffer_rsrc(routed ? p.ws + (size_t)tile.group * p.Nw * kb : p.wsh_s, clamp_bytes((size_t)p.Nw * kb));
        const __amdgpu_buffer_rsrc_t x_d =
            kGather ? buffer_rsrc(p.x, clamp_bytes((size_t)p.src.rows * rowb))
                    : buffer_rsrc(p.x + (size_t)tile.row0 * rowb, clamp_bytes((size_t)tile.rows * rowb));
        const __amdgpu_buffer_rsrc_t xs_d =
            kGather ? buffer_rsrc(p.xs, clamp_bytes((size_t)p.src.rows * kb))
                    : buffer_rsrc(p.xs + (size_t)tile.row0 * kb, clamp_bytes((size_t)tile.rows * kb));
        auto src_row = [&](int r) -> uint32_t {  // the tile's row r, clamped to it
            r = min(r, tile.rows - 1);
            if (!kGather) return (uint32_t)r;
            const int slot = p.src.row_slot[tile.row0 + r];
            const int t = slot < p.src.S ? slot / p.src.k : slot - p.src.S;
            return (uint32_t)max(0, min(t, p.src.rows - 1));
        };
        // piece 4i + wave of either operand holds LDS rows 16 (4i + wave) + [0, 16), four lanes a row. Piece
        // i's weight rows lie a uniform distance behind piece 0's.
        const int pr = 16 * wave + (lane >> 2);
        const uint32_t woff = (uint32_t)((kSwiGLU ? nb * 128 : nb * 256) + pr) * rowb + ((lane & 3) ^ mx_swz_w(pr)) * 16;
        auto wdist = [&](int i) -> uint32_t {
            return (uint32_t)(kSwiGLU ? (i < 2 ? 64 * i : I + 64 * (i - 2)) : 64 * i) * rowb;
        };
        uint32_t xoff[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) xoff[i] = src_row(64 * i + pr) * rowb + ((lane & 3) ^ mx_swz_x(pr)) * 16;
        // scales: wave w brings rows 64w + lane of both operands
        const uint32_t wsoff =
            (uint32_t)(kSwiGLU ? (wave >> 1) * I + nb * 128 + 64 * (wave & 1) : nb * 256 + 64 * wave) * kb + lane * kb;
        const uint32_t xsoff = src_row(64 * wave + lane) * kb;

        auto run = [&](auto nx_c) {
            constexpr int NX = decltype(nx_c)::value;
            auto issue = [&](int kc, MxStage& S) {  // steps past the end bring the last one again, unused
                const uint32_t ko = (uint32_t)min(kc, nk - 1) * kMxStepB;
#pragma unroll
                for (int i = 0; i < 4; ++i) lds_buf16(w_d, woff, wdist(i) + ko, &S.w[(4 * i + wave) * 1024]);
#pragma unroll
                for (int i = 0; i < NX; ++i) lds_buf16(x_d, xoff[i], ko, &S.x[(4 * i + wave) * 1024]);
            };
            auto issue_scales = [&](int kc) {
                const uint32_t so = (uint32_t)min(kc, nk - 1) / 4 * 16;
                lds_buf16(ws_d, wsoff, so, &sc.w[wave * 1024]);
                lds_buf16(xs_d, xsoff, so, &sc.x[wave * 1024]);
            };
            f32x16 acc[4][NX] = {};
            u32x4 sw[4], sx[NX];
            auto read_scales = [&]() {
#pragma unroll
                for (int s = 0; s < 4; ++s) sw[s] = *reinterpret_cast<const u32x4*>(&sc.w[(q0(s) + rw) * 16]);
#pragma unroll
                for (int j = 0; j < NX; ++j)
                    sx[j] = *reinterpret_cast<const u32x4*>(&sc.x[(64 * j + 32 * wm + l31) * 16]);
            };
            auto compute = [&](const MxStage& S, auto sub_c) {
                constexpr int sub = decltype(sub_c)::value;
                u32x4 a[4][2];
                uint32_t sa[4];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    sa[s] = sw[s][sub] >> (8 * hi);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        a[s][h] = *reinterpret_cast<const u32x4*>(&S.w[q0(s) * kMxStepB + offa[h]]);
                }
#pragma unroll
                for (int j = 0; j < NX; ++j) {
                    const u32x4 b0 = *reinterpret_cast<const u32x4*>(&S.x[j * 4096 + offb[0]]);
                    const u32x4 b1 = *reinterpret_cast<const u32x4*>(&S.x[j * 4096 + offb[1]]);
                    const uint32_t sb = sx[j][sub] >> (8 * hi);
#pragma unroll
                    for (int s = 0; s < 4; ++s) acc[s][j] = mfma_fp4<0, 0>(a[s][0], b0, acc[s][j], sa[s], sb);
#pragma unroll
                    for (int s = 0; s < 4; ++s) acc[s][j] = mfma_fp4<2, 2>(a[s][1], b1, acc[s][j], sa[s], sb);
                }
            };
            using C0 = std::integral_constant<int, 0>;
            using C1 = std::integral_constant<int, 1>;
            using C2 = std::integral_constant<int, 2>;
            using C3 = std::integral_constant<int, 3>;
            // loads of a step: 4 + NX, and two scale pieces ahead of every fourth
            constexpr int L = 4 + NX;
            issue_scales(0);
            issue(0, st0);
            issue(1, st1);
            issue(2, st2);
            for (int j = 0; j < nk; j += 4) {
                wait_vmcnt<2 * L>();  // step j and its scales have landed; j + 1 and j + 2 may fly
                barrier_only();
                issue(j + 3, st3);
                read_scales();
                compute(st0, C0{});
                wait_vmcnt<2 * L>();
                barrier_only();       // every wave holds the group's scales
                issue_scales(j + 4);
                issue(j + 4, st0);
                if (j + 1 < nk) compute(st1, C1{});
                wait_vmcnt<2 * L + 2>();
                barrier_only();
                issue(j + 5, st1);
                if (j + 2 < nk) compute(st2, C2{});
                wait_vmcnt<2 * L + 2>();
                barrier_only();
                issue(j + 6, st2);
                if (j + 3 < nk) compute(st3, C3{});
            }
            wait_vmcnt<0>();
            barrier_only();  // the ring is filled again by the next item

#pragma unroll
            for (int j = 0; j < NX; ++j) {
                const int m = 64 * j + 32 * wm + l31;
                const size_t row = (size_t)tile.row0 + m;
                if constexpr (kSwiGLU) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        float v[16];
                        uint32_t mx = 0;
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            v[r] = silu_mul(acc[s][j][r], acc[s + 2][j][r]);
                            mx = max(mx, abs_bits(v[r]));
                        }
                        mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32));
                        const uint32_t byte = mx_scale_byte(mx);
                        const float inv = mx_inverse(byte);
                        if (m < tile.rows) {
                            const int n0 = nb * 128 + 64 * wn + 32 * s;
                            *reinterpret_cast<uint2*>(p.out + row * (I / 2) + n0 / 2 + 8 * hi) =
                                make_uint2(mx_pack8(v, inv), mx_pack8(v + 8, inv));
                            if (hi == 0) p.out_scale[row * (I / kMxBlock) + n0 / kMxBlock] = (uint8_t)byte;
                        }
                    }
                } else if (m < tile.rows) {
                    uint16_t* y = reinterpret_cast<uint16_t*>(p.out) + row * p.Nw + nb * 256 + 128 * wn + 16 * hi;
#pragma unroll
                    for (int s = 0; s < 4; ++s)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const f32x16& a = acc[s][j];
                            *reinterpret_cast<u32x4*>(y + 32 * s + 8 * q) = u32x4{
                                pack_bf16x2(a[8 * q], a[8 * q + 1]), pack_bf16x2(a[8 * q + 2], a[8 * q + 3]),
                                pack_bf16x2(a[8 * q + 4], a[8 * q + 5]), pack_bf16x2(a[8 * q + 6], a[8 * q + 7])};
                        }
                }
            }
        };
        if (tile.rows <= 64)
            run(std::integral_constant<int, 1>{});
        else if (tile.rows <= 128)
            run(std::integral_constant<int, 2>{});
        else
            run(std::integral_constant<int, 4>{});
    }
}

// workspace: A codes [max_rows][I/2] | A scales [max_rows][I/32]
size_t mx_scale_offset(const moe_expert_weights* w, int max_rows) {
    return align_up((size_t)max_rows * (w->I / 2), 256);
}

template <bool kSwiGLU, bool kGather>
moe_status launch_gemm(const MxGemm& p, hipStream_t st) {
    const long tiles = (long)(p.max_rows + kMxTM - 1) / kMxTM + std::min(p.n_groups, p.max_rows);
    const int grid = (int)std::min((tiles * p.NB + 7) / 8 * 8, (long)device_info().cu_count / 8 * 8);
    hipLaunchKernelGGL((mx_gemm_kernel<kSwiGLU, kGather>), dim3(grid), dim3(kMxThreads), 0, st, p);
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
    p.NB = w->H / 256;
    p.out = (uint8_t*)y_perm;
    return launch_gemm<false, false>(p, st);
}

}  // namespace moe
