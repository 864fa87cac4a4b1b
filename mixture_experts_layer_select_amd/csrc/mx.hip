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

// Eight values a thread, a block in four neighbouring lanes. Bound by HBM: 4096 x
// 7168 fp32 take 27 us to quantise and 24 to read back (5.0 and 5.7 TB/s).
template <typename TIn>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const TIn* __restrict__ x, long n_eight,
                                                          uint32_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n_eight; i += (long)gridDim.x * 256) {
        float v[8];
        load_eight<TIn>(x + i * 8, v);
        uint32_t byte;
        codes[i] = mx_quantise8(v, byte);  // n_eight is a multiple of 4, so the four lanes run together
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
// workgroup of 8 waves per CU walks them (mx_item_at's order, a contiguous slice
// per XCD). Both operands of each K step of 256 (128 bytes of a row) arrive in
// LDS by direct global->LDS loads; the E8M0 scales of two steps come in one
// 16-byte piece per row and sit in registers for them. A load takes 8 rows of
// 128 bytes: 16 rows of 64 bytes moved 14 TB/s from L2 where these move 23.
// An item's first loads are issued before the previous item's epilogue.
//
// Measured at H = 7168, I = 2048, 32 experts, random codes (gate/up + down): 16
// rows an expert 96 + 57 us (5.2 and 4.4 TB/s of weights), 128 rows 125 + 76, 256
// rows 159 + 109, 512 rows 290 to 304 + 190 to 198 (3.2 and 2.5 PFLOP/s). From 256
// rows on the loads with one step in flight bound it: without the products they take
// 0.96 of the kernel's time on zero codes (0.86 with two steps in flight, for which
// LDS has no room), the products with their LDS reads alone 0.69.
//
// Waves form a 2 x 4 grid: wave (wm, wn) owns the 32-token blocks 2j + wm of
// the tile and 64 weight rows, as 2 x NX blocks of 32x32 accumulators, NX =
// 1 to 4 by the tile's height (64 rows each): a short tile loads only its own
// rows, so a group of up to 256 rows reads its weights from HBM once and
// little else. LDS holds two steps of a tile of more than 128 rows (64 KB
// each), or three of a shorter one, which HBM bounds (48 KB each).
//   SwiGLU: LDS rows q < 128 are gate rows nb*128 + q, q >= 128 the up rows I +
//     nb*128 + q - 128; wave wn owns gate q = 32wn + [0, 32) (s = 0) and the up
//     rows 128 + the same (s = 1).
//   Down: q -> w2 row nb*256 + q; wave wn owns q = 64wn + 32s + [0, 32).
// LDS rows are 128 bytes; chunk c of row q sits at chunk c ^ swz(q), which
// spreads the rows that 16 (and 8) consecutive lanes read over all banks.
constexpr int kMxTM = 256;     // tokens per tile
constexpr int kMxTN = 256;     // weight rows per tile
constexpr int kMxThreads = 512;
constexpr int kMxStepB = 128;  // bytes of a row per K step of 256
constexpr int kMxPanel = 4;    // m-tiles per item panel
constexpr int kKB = 1024;

struct MxScales {  // two K steps
    uint8_t w[kMxTN * 16];
    uint8_t x[kMxTM * 16];
};

// Tiles and rows of the groups, built by every workgroup once from the
// device-resident offsets: first tile (tile_start) and first row (row0, clamped
// to the buffer) of each group. A group's nt = ceil(m / height) tiles split its
// m rows evenly. Looked up from LDS alone, since every item's start waits for it.
constexpr int kMxMaxGroups = 513;  // E_local <= 512 and a shared group: checked by the C entry
struct MxTiles {
    int tile_start[kMxMaxGroups + 1];
    int row0[kMxMaxGroups + 1];
    int sums[3];
};

// All threads call (it holds barriers); returns the number of tiles. The height
// is 256 rows, or 128 or 64 where all items then still run at once: a call so
// small takes as long as its tallest tile (nine groups of 17 rows and one of 203
// at H = 1280, I = 384: gate/up 14.2 us with one tile of 203 rows, 10.0 with four).
__device__ __forceinline__ int mx_build_tiles(MxTiles& tm, const int32_t* __restrict__ offsets, int n_groups,
                                              int max_rows, int NB) {
    for (int g = threadIdx.x; g <= n_groups; g += kMxThreads) tm.row0[g] = clamp_row(offsets[g], max_rows);
    __syncthreads();
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int height = kMxTM >> wave;  // waves 0 to 2 count tiles of 256, 128 and 64 rows
    auto tiles_of = [&](int g, int h) {
        return g < n_groups ? max(0, tm.row0[g + 1] - tm.row0[g] + h - 1) / h : 0;
    };
    if (wave < 3) {
        int sum = 0;
        for (int g = lane; g < n_groups; g += 64) sum += tiles_of(g, height);
#pragma unroll
        for (int s = 32; s >= 1; s >>= 1) sum += __shfl_xor(sum, s);
        if (lane == 0) tm.sums[wave] = sum;
    }
    __syncthreads();
    const int h = tm.sums[2] <= (int)gridDim.x / NB ? 64 : tm.sums[1] <= (int)gridDim.x / NB ? 128 : kMxTM;
    if (wave == 0) {  // 64 groups at a time
        int run = 0;
        for (int g0 = 0; g0 < n_groups; g0 += 64) {
            const int g = g0 + lane, nt = tiles_of(g, h);
            int sum = nt;
#pragma unroll
            for (int s = 1; s < 64; s <<= 1) {
                const int o = __shfl_up(sum, s);
                if (lane >= s) sum += o;
            }
            if (g < n_groups) tm.tile_start[g] = run + sum - nt;
            run += __shfl(sum, 63);
        }
        if (lane == 0) tm.tile_start[n_groups] = run;
    }
    __syncthreads();
    return tm.tile_start[n_groups];
}

// Item -> tile and n-block, in panels of kMxPanel m-tiles of a group (the last
// one may be shorter): all n-blocks of a panel, its m-tiles fastest, so the
// workgroups of one XCD share both operands' slices of a K step through L2.
__device__ __forceinline__ MTile mx_item_at(const MxTiles& tm, int n_groups, int item, int NB, int& nb) {
    const int mt = item / NB;
    int lo = 0, hi = n_groups - 1;  // the group: the last g with tile_start[g] <= mt
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tm.tile_start[mid] <= mt) lo = mid;
        else hi = mid - 1;
    }
    const int t0 = __builtin_amdgcn_readfirstlane(tm.tile_start[lo]);
    const int nt = __builtin_amdgcn_readfirstlane(tm.tile_start[lo + 1]) - t0;
    const int r0 = __builtin_amdgcn_readfirstlane(tm.row0[lo]);
    const int m = __builtin_amdgcn_readfirstlane(tm.row0[lo + 1]) - r0;
    const int local = item - t0 * NB;
    const int pi = local / (kMxPanel * NB);  // never past the last panel
    const int ph = min(kMxPanel, nt - pi * kMxPanel);
    const int idx = local - pi * kMxPanel * NB;
    nb = idx / ph;
    const int i = pi * kMxPanel + idx - nb * ph;
    const int each = m / nt, more = m - each * nt;  // the first `more` tiles hold one row more
    return MTile{__builtin_amdgcn_readfirstlane(lo), r0 + i * each + min(i, more), each + (i < more ? 1 : 0)};
}

// weight row (within the wave's 32) that MFMA row rho reads: lane (l31, hi)
// then holds the D values of 16 consecutive weight rows 16 hi + [0, 16), so
// it writes 16 neighbouring outputs
__device__ __forceinline__ int mx_row_of(int rho) { return 16 * ((rho >> 2) & 1) + 4 * (rho >> 3) + (rho & 3); }
// chunk swizzles: weight rows are read in mx_row_of's order, tokens in rows'
__device__ __forceinline__ int mx_swz_w(int q) { return ((q & 3) ^ ((q >> 2) & 1)) | ((q >> 4) & 1) << 2; }
__device__ __forceinline__ int mx_swz_x(int q) { return (q & 7) ^ ((q >> 3) & 1); }

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
    // The stages are whole objects, or fixed parts of them, so that the compiler tells the ones being filled
    // from the one being read. Weights (32 KB) and tokens (16 KB for 128 rows) of a stage:
    //   two stages:   w o0, tokens 0-127 o0 + 32 KB, 128-255 o1 | w o2, tokens o3
    //   three stages: w o0, tokens o0 + 32 KB | w o2, tokens o1 | w o3, tokens o4
    __shared__ __attribute__((aligned(1024))) uint8_t o0[48 * kKB];
    __shared__ __attribute__((aligned(1024))) uint8_t o1[16 * kKB];
    __shared__ __attribute__((aligned(1024))) uint8_t o2[32 * kKB];
    __shared__ __attribute__((aligned(1024))) uint8_t o3[32 * kKB];
    __shared__ __attribute__((aligned(1024))) uint8_t o4[16 * kKB];
    __shared__ __attribute__((aligned(1024))) MxScales sc;
    __shared__ MxTiles tm;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int l31 = lane & 31, hi = lane >> 5;
    const int K = p.K, kb = K / kMxBlock, rowb = K / 2;
    const int nk = (K + 255) / 256;
    const int nk2 = K / 128;  // its halves: odd where the last step holds 128 of K
    const int I = p.Nw / 2;  // SwiGLU: intermediate size
    // uniform, so that the item loop and the descriptors it carries stay scalar
    const int n_items =
        __builtin_amdgcn_readfirstlane(mx_build_tiles(tm, p.offsets, p.n_groups, p.max_rows, p.NB)) * p.NB;
    const int xcd = blockIdx.x & 7;
    const int per_xcd = gridDim.x >> 3;
    const int i_lo = (int)((long)n_items * xcd / 8);
    const int i_hi = (int)((long)n_items * (xcd + 1) / 8);

    // fragment offsets in a stage: weight tile s at offa + q0(s) * 128, token block j at offb + j * 8192;
    // MFMA h of a step takes chunk 2h + hi of the row
    const int rw = mx_row_of(l31);
    int offa[4], offb[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        offa[h] = rw * kMxStepB + ((2 * h + hi) ^ mx_swz_w(rw)) * 16;
        offb[h] = (32 * wm + l31) * kMxStepB + ((2 * h + hi) ^ mx_swz_x(l31)) * 16;
    }
    auto q0 = [&](int s) MX_INLINE { return kSwiGLU ? 128 * s + 32 * wn : 64 * wn + 32 * s; };
    // piece 8i + wave of either operand holds LDS rows 64i + pr, eight lanes a row
    const int pr = 8 * wave + (lane >> 3);
    // a piece's weight rows lie a uniform distance behind piece 0's
    auto wdist = [&](int i) MX_INLINE -> uint32_t {
        return (uint32_t)(kSwiGLU ? (i < 2 ? 64 * i : I + 64 * (i - 2)) : 64 * i) * rowb;
    };

    // what an item's loads go by: its tile and this lane's offsets, and the descriptors, which are made anew
    // where they are used (carried through the item loop they would be kept in vector registers)
    struct Item {
        MTile tile;
        int nb;
        uint32_t woff, xoff[4], soff;
    };
    struct Desc {
        __amdgpu_buffer_rsrc_t w, x, s;
    };
    auto desc_of = [&](const MTile& t) MX_INLINE {
        const int group = __builtin_amdgcn_readfirstlane(t.group), row0 = __builtin_amdgcn_readfirstlane(t.row0),
                  rows = __builtin_amdgcn_readfirstlane(t.rows);
        const bool routed = group < p.n_routed;
        Desc d;
        d.w = buffer_rsrc(routed ? p.w + (size_t)group * p.Nw * rowb : p.wsh, clamp_bytes((size_t)p.Nw * rowb));
        d.x = kGather ? buffer_rsrc(p.x, clamp_bytes((size_t)p.src.rows * rowb))
                      : buffer_rsrc(p.x + (size_t)row0 * rowb, clamp_bytes((size_t)rows * rowb));
        // scales: waves 0..3 bring the weights', rows 64w + lane, waves 4..7 the tokens'
        if (wave < 4)
            d.s = buffer_rsrc(routed ? p.ws + (size_t)group * p.Nw * kb : p.wsh_s, clamp_bytes((size_t)p.Nw * kb));
        else
            d.s = kGather ? buffer_rsrc(p.xs, clamp_bytes((size_t)p.src.rows * kb))
                          : buffer_rsrc(p.xs + (size_t)row0 * kb, clamp_bytes((size_t)rows * kb));
        return d;
    };
    // An item in two parts: find() looks up its tile and asks for its rows' slots, place() makes the offsets from
    // them. The next item's find() stands ahead of the current one's steps, its place() behind them, so the slots
    // arrive under the products.
    const int w4 = wave & 3;
    auto find = [&](int item) MX_INLINE {
        Item c;
        c.tile = mx_item_at(tm, p.n_groups, item, p.NB, c.nb);
        auto slot = [&](int r) MX_INLINE -> uint32_t {  // of the tile's row r, clamped to it
            r = min(r, c.tile.rows - 1);
            return kGather ? (uint32_t)p.src.row_slot[c.tile.row0 + r] : (uint32_t)r;
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) c.xoff[i] = slot(64 * i + pr);
        c.soff = slot(64 * w4 + lane);
        return c;
    };
    auto place = [&](Item& c) MX_INLINE {
        auto src_row = [&](uint32_t v) MX_INLINE -> uint32_t {
            if (!kGather) return v;
            const int s = (int)v, tk = s < p.src.S ? s / p.src.k : s - p.src.S;
            return (uint32_t)max(0, min(tk, p.src.rows - 1));
        };
        c.woff = (uint32_t)((kSwiGLU ? c.nb * 128 : c.nb * 256) + pr) * rowb + ((lane & 7) ^ mx_swz_w(pr)) * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) c.xoff[i] = src_row(c.xoff[i]) * rowb + ((lane & 7) ^ mx_swz_x(pr)) * 16;
        c.soff = wave < 4
                     ? (uint32_t)((kSwiGLU ? (w4 >> 1) * I + c.nb * 128 + 64 * (w4 & 1) : c.nb * 256 + 64 * w4) + lane) * kb
                     : src_row(c.soff) * kb;
    };
    auto issue = [&](const Item& c, const Desc& d, auto nx_c, int kc, uint8_t* W, uint8_t* X01, uint8_t* X23) MX_INLINE {
        constexpr int NX = decltype(nx_c)::value;
        // Steps past the end, which the rings' counts include, bring the last one again, unused. (Loading nothing there,
        // from empty buffers, took 158.1 against 158.8 us at 128 decode tokens and 226.2 against 225.7 at 4096 while a
        // short tile still went six steps at a time; in the tall tiles' loop that test cost 6%.)
        const uint32_t ko = (uint32_t)min(kc, nk - 1) * kMxStepB;
#pragma unroll
        for (int i = 0; i < 4; ++i) lds_buf16(d.w, c.woff, wdist(i) + ko, W + (8 * i + wave) * 1024);
#pragma unroll
        for (int i = 0; i < NX; ++i)
            lds_buf16(d.x, c.xoff[i], ko, i < 2 ? X01 + (8 * i + wave) * 1024 : X23 + (8 * (i - 2) + wave) * 1024);
    };
    auto issue_scales = [&](const Item& c, const Desc& d, int kc) MX_INLINE {
        lds_buf16(d.s, c.soff, (uint32_t)min(kc, nk - 1) / 2 * 16, (wave < 4 ? sc.w : sc.x) + (wave & 3) * 1024);
    };
    auto with_nx = [&](int rows, auto f) MX_INLINE {
        if (rows <= 64) f(std::integral_constant<int, 1>{});
        else if (rows <= 128) f(std::integral_constant<int, 2>{});
        else if (rows <= 192) f(std::integral_constant<int, 3>{});
        else f(std::integral_constant<int, 4>{});
    };
    auto first_loads = [&](const Item& c) MX_INLINE {
        const Desc d = desc_of(c.tile);
        issue_scales(c, d, 0);
        with_nx(__builtin_amdgcn_readfirstlane(c.tile.rows), [&](auto nx_c) MX_INLINE {
            if constexpr (decltype(nx_c)::value > 2) {
                issue(c, d, nx_c, 0, o0, o0 + 32 * kKB, o1);
            } else {
                issue(c, d, nx_c, 0, o0, o0 + 32 * kKB, nullptr);
                asm volatile("" ::: "memory");  // in this order: the waits count the loads
                issue(c, d, nx_c, 1, o2, o1, nullptr);
            }
        });
    };

    int item = i_lo + (int)(blockIdx.x >> 3);
    if (item >= i_hi) return;
    Item cur = find(item);
    place(cur);
    first_loads(cur);
    for (;;) {
        const bool more = item + per_xcd < i_hi;
        Item next = more ? find(item + per_xcd) : cur;
        const MTile tile{__builtin_amdgcn_readfirstlane(cur.tile.group), __builtin_amdgcn_readfirstlane(cur.tile.row0),
                         __builtin_amdgcn_readfirstlane(cur.tile.rows)};
        const int nb = __builtin_amdgcn_readfirstlane(cur.nb);
        const Desc d = desc_of(tile);
        auto run = [&](auto nx_c) MX_INLINE {
            constexpr int NX = decltype(nx_c)::value;
            f32x16 acc[2][NX] = {};
            u32x4 sw[2], sx[NX];
            auto read_scales = [&]() MX_INLINE {
#pragma unroll
                for (int s = 0; s < 2; ++s) sw[s] = *reinterpret_cast<const u32x4*>(&sc.w[(q0(s) + rw) * 16]);
#pragma unroll
                for (int j = 0; j < NX; ++j)
                    sx[j] = *reinterpret_cast<const u32x4*>(&sc.x[(64 * j + 32 * wm + l31) * 16]);
            };
            // step kc from a stage; sub: its two dwords of the group's scales
            auto compute = [&](int kc, auto sub_c, const uint8_t* W, const uint8_t* X01, const uint8_t* X23) MX_INLINE {
                constexpr int sub = decltype(sub_c)::value;
                auto part = [&](auto u_c) MX_INLINE {  // 128 of K: MFMAs h = 2u, 2u + 1
                    constexpr int u = decltype(u_c)::value;
                    // the half past an odd end multiplies by scales of 2^-127
                    const uint32_t on = 2 * kc + u < nk2 ? ~0u : 0u;
                    u32x4 a[2][2];
                    uint32_t sa[2];
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        sa[s] = (sw[s][2 * sub + u] >> (8 * hi)) & on;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            a[s][h] = *reinterpret_cast<const u32x4*>(W + q0(s) * kMxStepB + offa[2 * u + h]);
                    }
#pragma unroll
                    for (int j = 0; j < NX; ++j) {
                        const uint8_t* X = j < 2 ? X01 + j * 8192 : X23 + (j - 2) * 8192;
                        const u32x4 b0 = *reinterpret_cast<const u32x4*>(X + offb[2 * u]);
                        const u32x4 b1 = *reinterpret_cast<const u32x4*>(X + offb[2 * u + 1]);
                        const uint32_t sb = (sx[j][2 * sub + u] >> (8 * hi)) & on;
#pragma unroll
                        for (int s = 0; s < 2; ++s) acc[s][j] = mfma_fp4<0, 0>(a[s][0], b0, acc[s][j], sa[s], sb);
#pragma unroll
                        for (int s = 0; s < 2; ++s) acc[s][j] = mfma_fp4<2, 2>(a[s][1], b1, acc[s][j], sa[s], sb);
                    }
                };
                part(std::integral_constant<int, 0>{});
                part(std::integral_constant<int, 1>{});
            };
            using C0 = std::integral_constant<int, 0>;
            using C1 = std::integral_constant<int, 1>;
            // A group's scales are issued in its last step but one, after the barrier behind which every wave
            // holds the previous group's, and ahead of that step's own loads, so each wait below covers them.
            if constexpr (NX > 2) {
                auto S0 = [&](auto f) MX_INLINE { f(o0, o0 + 32 * kKB, o1); };
                auto S1 = [&](auto f) MX_INLINE { f(o2, o3, o3 + 16 * kKB); };
                auto load = [&](int kc, auto at) MX_INLINE {
                    at([&](uint8_t* W, uint8_t* X01, uint8_t* X23) MX_INLINE { issue(cur, d, nx_c, kc, W, X01, X23); });
                };
                auto work = [&](int kc, auto sub, auto at) MX_INLINE {
                    at([&](uint8_t* W, uint8_t* X01, uint8_t* X23) MX_INLINE { compute(kc, sub, W, X01, X23); });
                };
                for (int j = 0; j < nk; j += 2) {
                    wait_vmcnt<0>();
                    mx_barrier();
                    load(j + 1, S1);
                    read_scales();
                    work(j, C0{}, S0);
                    wait_vmcnt<0>();
                    mx_barrier();
                    issue_scales(cur, d, j + 2);
                    load(j + 2, S0);
                    if (j + 1 < nk) work(j + 1, C1{}, S1);
                }
            } else {
                constexpr int L = 4 + NX;  // a step's loads
                auto S0 = [&](auto f) MX_INLINE { f(o0, o0 + 32 * kKB); };
                auto S1 = [&](auto f) MX_INLINE { f(o2, o1); };
                auto S2 = [&](auto f) MX_INLINE { f(o3, o4); };
                auto load = [&](int kc, auto at) MX_INLINE {
                    at([&](uint8_t* W, uint8_t* X) MX_INLINE { issue(cur, d, nx_c, kc, W, X, nullptr); });
                };
                auto work = [&](int kc, auto sub, auto at) MX_INLINE {
                    at([&](uint8_t* W, uint8_t* X) MX_INLINE { compute(kc, sub, W, X, nullptr); });
                };
                auto even = [&](int j, auto cur_s, auto next_s) MX_INLINE {
                    wait_vmcnt<L>();  // step j and its scales have landed; j + 1 may fly
                    mx_barrier();
                    load(j + 2, next_s);
                    if (j < nk) {
                        read_scales();
                        work(j, C0{}, cur_s);
                    }
                };
                auto odd = [&](int j, auto cur_s, auto next_s) MX_INLINE {
                    wait_vmcnt<L>();
                    mx_barrier();
                    issue_scales(cur, d, j + 1);
                    asm volatile("" ::: "memory");  // in this order: the waits count the loads
                    load(j + 2, next_s);
                    if (j < nk) work(j, C1{}, cur_s);
                };
                for (int j = 0; j < nk; j += 6) {
                    even(j, S0, S2);
                    odd(j + 1, S1, S0);
                    if (j + 2 >= nk) break;  // at most three steps past the end: 158.7 -> 151.3 us at 128 decode tokens
                    even(j + 2, S2, S1);
                    odd(j + 3, S0, S2);
                    if (j + 4 >= nk) break;
                    even(j + 4, S1, S0);
                    odd(j + 5, S2, S1);
                }
            }
            wait_vmcnt<0>();
            mx_barrier();  // no stage is read any more
            if (more) {
                place(next);
                first_loads(next);
            }

#pragma unroll
            for (int j = 0; j < NX; ++j) {
                const int m = 64 * j + 32 * wm + l31;
                const size_t row = (size_t)tile.row0 + m;
                if constexpr (kSwiGLU) {
                    float v[16];
                    uint32_t mx = 0;
                    // With the divide, as moe_layer_few has it: a reciprocal instruction gives 0 where exp(-g) is above
                    // 2^126, and its last bit moved codes (9 rows of 165 000 against the plain form, 3 with the divide; none
                    // with expf, for 2% at 16384 tokens). It costs 1 us at 128 decode tokens, 2 at 4096, 10 at 16384.
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        v[r] = silu_mul(acc[0][j][r], acc[1][j][r]);
                        mx = max(mx, abs_bits(v[r]));
                    }
                    mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32));
                    const uint32_t byte = mx_scale_byte(mx);
                    const float inv = mx_inverse(byte);
                    if (m < tile.rows) {
                        const int n0 = nb * 128 + 32 * wn;
                        *reinterpret_cast<uint2*>(p.out + row * (I / 2) + n0 / 2 + 8 * hi) =
                            make_uint2(mx_pack8(v, inv), mx_pack8(v + 8, inv));
                        if (hi == 0) p.out_scale[row * (I / kMxBlock) + n0 / kMxBlock] = (uint8_t)byte;
                    }
                } else if (m < tile.rows) {
                    uint16_t* y = reinterpret_cast<uint16_t*>(p.out) + row * p.Nw + nb * 256 + 64 * wn + 16 * hi;
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const f32x16& a = acc[s][j];
                            *reinterpret_cast<u32x4*>(y + 32 * s + 8 * q) = u32x4{
                                cvt_bf16x2(a[8 * q], a[8 * q + 1]), cvt_bf16x2(a[8 * q + 2], a[8 * q + 3]),
                                cvt_bf16x2(a[8 * q + 4], a[8 * q + 5]), cvt_bf16x2(a[8 * q + 6], a[8 * q + 7])};
                        }
                }
            }
        };
        with_nx(tile.rows, run);
        if (!more) break;
        item += per_xcd;
        cur = next;
    }
}

// workspace: A codes [max_rows][I/2] | A scales [max_rows][I/32]
size_t mx_scale_offset(const moe_expert_weights* w, int max_rows) {
    return align_up((size_t)max_rows * (w->I / 2), 256);
}

template <bool kSwiGLU, bool kGather>
moe_status launch_gemm(const MxGemm& p, hipStream_t st) {
    const long tiles = ((long)p.max_rows + 63) / 64 + std::min(p.n_groups, p.max_rows);  // of 64 rows, at most
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
