// Matrix products grouped by expert, for training: an expert's rows through its
// weights, the gradient of those rows, and the gradient of the weights. The rows
// of group g are [offsets[g], offsets[g + 1]), on the device.
//
//   forward  y[r, n]     = sum_k x[r, k]  w[g, n, k]    contraction over k
//   input    dx[r, k]    = sum_n dy[r, n] w[g, n, k]    over n
//   weights  dw[g, n, k] = sum_r dy[r, n] x[r, k]       over the group's rows
//
// In each, P is the operand that runs along the output's columns (w, w, x) and
// Q the one along its rows (x, dy, dy). An operand is stored with the
// contraction along its rows ("K-contiguous": both of forward, Q of input) or
// down its columns ("K-strided": P of input, both of weights).
#include "mx_dev.h"
#include "tile_dev.h"

namespace moe {
namespace {

enum Form { kForward = 0, kInput = 1, kWeights = 2 };

struct GemmArgs {
    const void *p, *p_last;  // w of the routed groups and of the last one (null: there is none apart); x rows for kWeights
    const void* q;           // x, dy, dy
    const int32_t* offsets;
    int n_groups, max_rows, N, K;
    void *out, *out_last;  // kWeights: dw of the routed groups and of the last one
    int accumulate;
    int height;  // kWeights: rows of a tile, 64 to 256
};

// ============================================================================ fp32
// Tiles of 64 x 64, 4 waves of a quarter each, operands through registers into
// two LDS stages, loads kAhead steps ahead. A step takes kStep of the
// contraction: of each row of a K-contiguous operand, or kStep rows of a
// K-strided one. Bound by the matrix cores (an fp32 product costs sixteen bf16
// ones), so blocks past a tile's rows are left out. 4096 rows of 8 groups, 2048 x
// 2048: 350 us forward and input (98 TFLOP/s), 320 weights, with steps of 16;
// tiles of 128 took 408, 408 and 283, steps of 32 390, 388 and 333.
//
// Calls of few tiles are as long as their chain of steps: they take steps of 32,
// and in a tile of at most 32 rows the two waves that would have none take
// the second half of each step, their sums joined at the end. 203 rows of 9
// groups, 768 x 1280: forward 25 us, input 18, against 38 and 26; 200 rows of 32
// groups, 1000 x 1000: 25 and 31, against 32 and 34.
constexpr int kT = 64;
constexpr int kAhead = 2;    // four: the same
constexpr int kF32Grid = 4;  // workgroups per CU; eight for dw, whose items are short (320 -> 308 us, others slower)
template <int kStep>
struct F32Step {
    static constexpr int row_c = kStep * 4 + 16;  // LDS bytes of a K-contiguous row
    static constexpr int row_s = kT * 4 + 16;     // and of a K-strided one
    static constexpr int bytes = kT * row_c > kStep * row_s ? kT * row_c : kStep * row_s;
    static constexpr int pieces = kStep / 16;     // 16-byte pieces of an operand that a thread loads
    struct Regs {
        u32x4 v[pieces];
    };
};

// Where this thread's piece i of a step's operand tile lies: output index and place in the contraction.
template <int kStep, bool kContig>
__device__ __forceinline__ int piece_o(int i) {
    return kContig ? (threadIdx.x + 256 * i) / (kStep / 4) : threadIdx.x % (kT / 4) * 4;
}
template <int kStep, bool kContig>
__device__ __forceinline__ int piece_k(int i) {
    return kContig ? (threadIdx.x & (kStep / 4 - 1)) * 4 : threadIdx.x / (kT / 4) + 16 * i;
}
// What lies outside the operand is loaded from its edge, without branches, and staged as zeros.
template <int kStep, bool kContig>
__device__ __forceinline__ typename F32Step<kStep>::Regs fetch(const float* base, size_t ld, int n_out, int out0, int n_k,
                                                               int k0) {
    typename F32Step<kStep>::Regs r;
#pragma unroll
    for (int i = 0; i < F32Step<kStep>::pieces; ++i) {
        const int o = min(out0 + piece_o<kStep, kContig>(i), n_out - (kContig ? 1 : 4));
        const int k = min(k0 + piece_k<kStep, kContig>(i), n_k - (kContig ? 4 : 1));
        r.v[i] = *reinterpret_cast<const u32x4*>(base + (kContig ? (size_t)o * ld + k : (size_t)k * ld + o));
    }
    return r;
}
template <int kStep, bool kContig>
__device__ __forceinline__ void stage(uint8_t* l, int n_out, int out0, int n_k, int k0,
                                      const typename F32Step<kStep>::Regs& r) {
    using S = F32Step<kStep>;
#pragma unroll
    for (int i = 0; i < S::pieces; ++i) {
        const int o = piece_o<kStep, kContig>(i), k = piece_k<kStep, kContig>(i);
        const bool in = out0 + o < n_out && k0 + k < n_k;
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = in ? r.v[i][e] : 0u;
        *reinterpret_cast<u32x4*>(l + (kContig ? o * S::row_c + k * 4 : k * S::row_s + o * 4)) = v;
    }
}
// lane (li, lk) of a 16-wide block at output o0: elements 16 h + 4 lk + [0, 4) of the step's contraction
template <int kStep, bool kContig>
__device__ __forceinline__ f32x4 fragment(const uint8_t* l, int o0, int h, int li, int lk) {
    using S = F32Step<kStep>;
    if constexpr (kContig) {
        return *reinterpret_cast<const f32x4*>(l + (o0 + li) * S::row_c + h * 64 + lk * 16);
    } else {
        f32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = *reinterpret_cast<const float*>(l + (16 * h + lk * 4 + j) * S::row_s + (o0 + li) * 4);
        return v;
    }
}

template <int kForm, int kStep>
__global__ __launch_bounds__(256, kStep == 16 ? kF32Grid : 2) void gemm_f32_kernel(GemmArgs a) {
    using S = F32Step<kStep>;
    constexpr bool kPc = kForm == kForward, kQc = kForm != kWeights;
    constexpr int kB = kT / 32;  // 16-wide blocks of a wave, each way
    __shared__ __attribute__((aligned(16))) uint8_t lp[2][S::bytes], lq[2][S::bytes];
    __shared__ RowTiles<kMaxGroups> tm;
    const int lane = threadIdx.x & 63, li = lane & 15, lk = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = wave >> 1;
    const int wp = (wave & 1) * (kT / 2);
    const int cols = kForm == kForward ? a.N : a.K;  // of the output
    const int NB = (cols + kT - 1) / kT, MB = (a.N + kT - 1) / kT;
    const size_t w_size = (size_t)a.N * a.K, ldq = kForm == kForward ? a.K : a.N;
    const bool apart = kForm == kWeights ? a.out_last != nullptr : a.p_last != nullptr;
    int n_items;
    if constexpr (kForm == kWeights) n_items = a.n_groups * MB * NB;
    else n_items = even_tiles<256>(tm, a.offsets, a.n_groups, a.max_rows, kT) * NB;

    for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
        const float *p, *q;
        float* out;
        int nb, q0, rows, n_k;  // column block; first output row, rows that end the tile, length of the contraction
        if constexpr (kForm == kWeights) {
            const int g = item / (MB * NB), in = item % (MB * NB);
            const int r0 = clamp_row(a.offsets[g], a.max_rows), r1 = clamp_row(a.offsets[g + 1], a.max_rows);
            nb = in % NB;
            q0 = in / NB * kT;
            rows = a.N;
            n_k = max(0, r1 - r0);
            p = (const float*)a.p + (size_t)r0 * a.K;
            q = (const float*)a.q + (size_t)r0 * a.N;
            out = apart && g == a.n_groups - 1 ? (float*)a.out_last : (float*)a.out + g * w_size;
        } else {
            const MTile t = row_item_at(tm, a.n_groups, item, NB, nb);
            n_k = kForm == kForward ? a.K : a.N;
            p = apart && t.group == a.n_groups - 1 ? (const float*)a.p_last : (const float*)a.p + t.group * w_size;
            q = (const float*)a.q + (size_t)t.row0 * n_k;
            out = (float*)a.out + (size_t)t.row0 * cols;
            q0 = 0;
            rows = t.rows;
        }
        const bool split = kStep == 32 && rows - q0 <= kT / 2;
        const int wq = split ? 0 : half * (kT / 2);
        const int nj = (rows - q0 - wq + 15) / 16;  // of this wave's row blocks, those that hold rows
        f32x4 acc[kB][kB] = {};
        typename S::Regs rp[kAhead], rq[kAhead];
        const int nk = (n_k + kStep - 1) / kStep;
        auto load = [&](int kc, int s) {
            rp[s] = fetch<kStep, kPc>(p, a.K, cols, nb * kT, n_k, kc * kStep);
            rq[s] = fetch<kStep, kQc>(q, ldq, rows, q0, n_k, kc * kStep);
        };
        auto put = [&](int kc, int s) {
            stage<kStep, kPc>(lp[kc & 1], cols, nb * kT, n_k, kc * kStep, rp[s]);
            stage<kStep, kQc>(lq[kc & 1], rows, q0, n_k, kc * kStep, rq[s]);
        };
        __syncthreads();  // the previous item's reads
        if (nk > 0) {
#pragma unroll
            for (int s = 0; s < kAhead; ++s) load(s, s);  // steps past the end load the edge again, unused
            put(0, 0);
            load(kAhead, 0);
        }
        for (int k0 = 0; k0 < nk; k0 += kAhead) {
#pragma unroll
            for (int s = 0; s < kAhead; ++s) {
                const int kc = k0 + s;
                if (kc >= nk) break;
                barrier_only();  // step kc is staged; the loads ahead stay in flight
#pragma unroll
                for (int h = 0; h < kStep / 16; ++h) {
                    if (split && h != half) continue;
                    f32x4 fp[kB], fq[kB];
#pragma unroll
                    for (int i = 0; i < kB; ++i) {
                        fp[i] = fragment<kStep, kPc>(lp[kc & 1], wp + 16 * i, h, li, lk);
                        fq[i] = fragment<kStep, kQc>(lq[kc & 1], wq + 16 * i, h, li, lk);
                    }
#pragma unroll
                    for (int j = 0; j < kB; ++j)
                        if (j < nj) {
#pragma unroll
                            for (int t = 0; t < 4; ++t)
#pragma unroll
                                for (int i = 0; i < kB; ++i)
                                    acc[i][j] =
                                        __builtin_amdgcn_mfma_f32_16x16x4f32(fp[i][t], fq[j][t], acc[i][j], 0, 0, 0);
                        }
                }
                put(kc + 1, (s + 1) % kAhead);  // the other stage: its readers passed this step's barrier
                load(kc + 1 + kAhead, (s + 1) % kAhead);
            }
        }
        if (split) {
            __syncthreads();  // the last step's reads
            f32x4* sums = reinterpret_cast<f32x4*>(lp[0]) + (wave & 1) * 64 * kB * kB;
            static_assert(2 * 64 * kB * kB * 16 <= 2 * S::bytes, "the second halves' sums lie in P's stages");
#pragma unroll
            for (int n = 0; n < kB * kB; ++n)
                if (half == 1) sums[n * 64 + lane] = acc[n / kB][n % kB];
            __syncthreads();
            if (half == 1) continue;
#pragma unroll
            for (int n = 0; n < kB * kB; ++n) acc[n / kB][n % kB] += sums[n * 64 + lane];
        }
        // lane (li, lk): columns 4 lk + [0, 4) of the block at output row li
        if (kForm == kWeights && nk == 0 && a.accumulate) continue;
#pragma unroll
        for (int j = 0; j < kB; ++j) {
            const int r = q0 + wq + 16 * j + li;
#pragma unroll
            for (int i = 0; i < kB; ++i) {
                const int c = nb * kT + wp + 16 * i + 4 * lk;
                if (r < rows && c < cols) {
                    f32x4* o = reinterpret_cast<f32x4*>(out + (size_t)r * cols + c);
                    *o = a.accumulate ? acc[i][j] + *o : acc[i][j];
                }
            }
        }
    }
}

template <int kForm>
moe_status launch_f32(const GemmArgs& a, hipStream_t st) {
    const long nb = ((kForm == kForward ? a.N : a.K) + kT - 1) / kT;
    const long tiles = kForm == kWeights ? (long)a.n_groups * ((a.N + kT - 1) / kT)
                                         : ((long)a.max_rows + kT - 1) / kT + std::min(a.n_groups, a.max_rows);
    const int grid = (int)std::min(tiles * nb, (long)device_info().cu_count * (kForm == kWeights ? 8 : kF32Grid));
    if constexpr (kForm != kWeights) {
        if (tiles * nb <= (long)device_info().cu_count * kF32Grid) {  // all at once
            hipLaunchKernelGGL((gemm_f32_kernel<kForm, 32>), dim3(grid), dim3(256), 0, st, a);
            return check_launch("gemm_f32_kernel");
        }
    }
    hipLaunchKernelGGL((gemm_f32_kernel<kForm, 16>), dim3(grid), dim3(256), 0, st, a);
    return check_launch("gemm_f32_kernel");
}

// ============================================================================ bf16, an LDS ring
// Tiles of up to 256 x 256 on 8 waves, one workgroup a CU: wave (wm, wn) of a 2 x 4 grid owns the 32-row blocks
// 2j + wm and 64 columns, as 2 x NX blocks of 32 x 32 accumulators (NX = 1 to 4 by the tile's height). Both operands
// of a step arrive in LDS by direct loads, a ring of steps ahead of the products; XCDs walk contiguous slices of the
// items (row_item_at's order), so that tiles that run side by side share operands through L2.
//
// K-contiguous operands lie in rows of 128 bytes and are read 16 bytes a lane; K-strided ones in rows of 512 (256
// columns of one row) and are read transposed: ds_read_b64_tr_b16 hands lane i of sixteen the
// element i of four rows, and two such reads make its eight of the contraction. The swizzles spread both over the
// banks (no conflicts counted).
//
// A step's barrier stands before its last quarter, whose fragments are in registers by then, so no wave waits at it
// with idle matrix cores; the loads of a later step stand one behind each pair of products. In a burst behind the
// barrier they kept waves from issuing products (one group of 8192^3, forward: 911 us; spread 836, and 801 with the
// ring's rest behind its loop). There it runs at 1.37 PFLOP/s, dx at 1.40 and dw at 1.31, with a clock that falls to 1.4 to
// 1.6 GHz under the products; a large library product of the same layouts reaches 1.39, 1.23 and 1.08.
constexpr int kBig = 256;  // rows and columns of a tile
constexpr int kBigThreads = 512;
constexpr int kNonTemporal = 2;  // buffer stores' cache policy

typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x4 lds_read_tr(const uint8_t* l) {
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(l));
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(l + 2048));
    const uint2 u = __builtin_bit_cast(uint2, x), v = __builtin_bit_cast(uint2, y);
    return u32x4{u.x, u.y, v.x, v.y};
}
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}
// Column (within 32) that MFMA row rho computes: a lane then holds 8 (bf16) or 4 (fp32) neighbouring columns a 16-byte
// store, and its neighbour at lane + 32 the next ones.
template <typename TO>
__device__ __forceinline__ int col_of(int rho) {
    return sizeof(TO) == 4 ? rho : 16 * (rho >> 4) + 8 * ((rho >> 2) & 1) + 4 * ((rho >> 3) & 1) + (rho & 3);
}
// chunk swizzles: of rows of 128 bytes read in col_of's order and in order, of rows of 512 read transposed
template <typename TO>
__device__ __forceinline__ int swz_p(int q) {
    return sizeof(TO) == 4 ? (q & 7) ^ ((q >> 3) & 1) : ((q & 3) | ((q >> 3) & 1) << 2) ^ ((q >> 2) & 1);
}
__device__ __forceinline__ int swz_q(int q) { return (q & 7) ^ ((q >> 3) & 1); }
__device__ __forceinline__ int swz_k(int r) { return (r & 3) | ((r >> 3) & 1) << 2; }

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t old, float lo, float hi) {
    return cvt_bf16x2(lo + bf16_lo(old), hi + bf16_hi(old));
}
// sixteen values of a lane, to columns c0 + [0, 32) of an output row
__device__ __forceinline__ void put16(uint16_t* o, int c0, int cols, int hi, const f32x16& v, bool add) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int c = c0 + 16 * t + 8 * hi;
        if (c >= cols) continue;
        u32x4* p = reinterpret_cast<u32x4*>(o + c);
        u32x4 w;
        if (add) {
            const u32x4 old = *p;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = add_bf16x2(old[i], v[8 * t + 2 * i], v[8 * t + 2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = cvt_bf16x2(v[8 * t + 2 * i], v[8 * t + 2 * i + 1]);
        }
        *p = w;
    }
}
__device__ __forceinline__ void put16(float* o, int c0, int cols, int hi, const f32x16& v, bool add) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int c = c0 + 8 * t + 4 * hi;
        if (c >= cols) continue;
        f32x4* p = reinterpret_cast<f32x4*>(o + c);
        f32x4 w = {v[4 * t], v[4 * t + 1], v[4 * t + 2], v[4 * t + 3]};
        if (add) w += *p;
        *p = w;
    }
}

// Stores of a bf16 tile. A lane holds a row's columns in four runs of eight, which change places within its quad of lanes
// (four rows), so that eight lanes' 16-byte stores make a line of 128 bytes (16384 rows of 32 experts, gradient of
// 7168 x 4096 weights: 1132 us with half sectors of 32 rows a store, 1047 so, 1030 past L2).
template <int kCtrl>
__device__ __forceinline__ uint32_t quad_perm(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xf, 0xf, false);
}
// register k of lane i of a quad <- register i of lane k
__device__ __forceinline__ u32x4 quad_transpose(u32x4 a, int i) {
    const bool b0 = i & 1, b1 = i & 2;
    const uint32_t p0 = quad_perm<0xb1>(a[0]), p1 = quad_perm<0xb1>(a[1]), p2 = quad_perm<0xb1>(a[2]),
                   p3 = quad_perm<0xb1>(a[3]);  // all lanes take part: outside the selects
    const u32x4 t = {b0 ? p1 : a[0], b0 ? a[1] : p0, b0 ? p3 : a[2], b0 ? a[3] : p2};
    const uint32_t q0 = quad_perm<0x4e>(t[0]), q1 = quad_perm<0x4e>(t[1]), q2 = quad_perm<0x4e>(t[2]),
                   q3 = quad_perm<0x4e>(t[3]);
    return u32x4{b1 ? q2 : t[0], b1 ? q3 : t[1], b1 ? t[2] : q0, b1 ? t[3] : q1};
}
// rows m0 + [0, 32) (this lane's: m0 + l31) and columns c0 + [0, 64) of an output with rows of `ld`, of which `rows` rows
// (in the descriptor) and `cols` columns are kept
__device__ __forceinline__ void put_block(__amdgpu_buffer_rsrc_t d, int ld, int m0, int c0, int cols, int lane,
                                          const f32x16& a0, const f32x16& a1) {
    const int i4 = lane & 3, hi = lane >> 5;
    u32x4 x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const u32x4 v = quad_transpose(u32x4{cvt_bf16x2(a0[2 * e], a0[2 * e + 1]), cvt_bf16x2(a0[8 + 2 * e], a0[9 + 2 * e]),
                                             cvt_bf16x2(a1[2 * e], a1[2 * e + 1]), cvt_bf16x2(a1[8 + 2 * e], a1[9 + 2 * e])},
                                       i4);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k][e] = v[k];
    }
    const int c = c0 + 16 * i4 + 8 * hi;
    const uint32_t at = c < cols ? ((uint32_t)(m0 + (lane & 28)) * ld + c) * 2 : 0x40000000u;
#pragma unroll
    for (int k = 0; k < 4; ++k) __builtin_amdgcn_raw_buffer_store_b128(x[k], d, at + 2u * k * ld, 0, kNonTemporal);
}

// ---------------------------------------------------------------- rows: forward and input
// Which tiles a call is cut into: every workgroup finds the same plan from the
// device-resident offsets. A group's m rows split evenly into ceil(m / height)
// tiles, the columns into blocks of `width`. Looked up from LDS alone, since
// every item's start waits for it.
struct RowsPlan {
    RowTiles<kMaxGroups> t;
    uint32_t cost[4];  // of the best width for each height
    int tiles[4], width[4];
};

// of whole numbers, for the estimate only; the division rounds correctly, so a whole quotient stays whole
__device__ __forceinline__ float ceil_div(float a, float b) { return ceilf(a / b); }

// All threads call; returns the number of tiles, their height and the column blocks' width. Of the heights 64 to 256 and
// the widths 64 to 256 (multiples of kUnit; of 64 where the products bound it, since a wave's 64 columns cost the same
// whether they are there or not) it takes the pair with the shortest estimate: the rounds of items that a workgroup
// walks, times a step's time, times the steps and three for an item's start and end. A step of a tile of h x w columns
// takes about 0.2 + 0.3 NX + (0.4 + 0.65 / mt) w / 256 us, NX = ceil(h / 64), mt tiles of a group sharing the weights:
// 0.2 NX up to 128 columns (four waves of eight have products), the loads' term down to half where few CUs load. Tiles
// of 64 x 64 split their contraction over the waves: a quarter of the steps, with the loads of a whole tile
// (K-strided P in pieces of 128 bytes of a row instead of 512: 1.35 times as long where rounds follow one another).
// All sixteen pairs of 64, 128, 192 and 256 were timed on 30 calls of 50 to 16384 rows and 300 to 7168 columns: the
// plan's pair takes 1% longer than the fastest in the mean, 10% at most. Every workgroup waits for the search, about 1 us
// of a call: sums by DPP moves, quotients in fp32 instead of integer divisions, and one minimum that carries its lane
// (50 rows of 16 groups, 1000 x 1000, forward: 9.9 -> 9.3 us; 100 rows of 8 groups, 2000 x 296: 8.7 -> 7.8).
template <int kUnit>
__device__ __forceinline__ int plan_rows(RowsPlan& plan, const int32_t* __restrict__ offsets, int n_groups,
                                         int max_rows, int cols, int nk, int& width,
                                         int& height) {
    for (int g = threadIdx.x; g <= n_groups; g += kBigThreads) plan.t.row0[g] = clamp_row(offsets[g], max_rows);
    __syncthreads();
    constexpr float kSplitLoads = kUnit == 64 ? 1.35f : 1.0f;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (wave < 4) {
        const int parts = wave + 1, h = 64 * parts;
        int tiles = 0;
        float nx = 0.f, share = 0.f;  // summed over the tiles: 64-row pieces, and parts of a group's weights
        for (int g = lane; g < n_groups; g += 64) {
            const int q = (max(0, plan.t.row0[g + 1] - plan.t.row0[g]) + 63) >> 6;  // pieces of 64 rows
            const int nt = parts == 1 ? q : parts == 2 ? (q + 1) >> 1 : parts == 3 ? (q + 2) / 3 : (q + 3) >> 2;
            if (nt) {
                tiles += nt;
                nx += (float)nt * ceil_div((float)q, (float)nt);
                share += 1.0f;
            }
        }
        tiles = wave_total(tiles);
        nx = wave_total(nx);
        share = wave_total(share);
        const int w = kBig - kUnit * lane;
        // the estimate's bits, the lane in the lowest six: the smallest is the best width's (positive floats sort as integers)
        uint32_t cost = 0x7f000000u + lane;
        if (w >= 64 && tiles && (w % 64 == 0 || nx <= 2.0f * (float)tiles)) {
            const float items = (float)tiles * ceil_div((float)cols, (float)w);
            const float rounds = ceil_div(ceilf(0.125f * items), (float)(gridDim.x >> 3));
            const bool split = h == 64 && w == 64;
            const float part = !split ? (float)w / kBig : rounds > 1.f ? kSplitLoads : 1.0f, each = 1.0f / (float)tiles;
            const float busy = fminf(1.0f, items / (float)gridDim.x);
            const float step = 0.2f + nx * each * (w <= 128 ? 0.2f : 0.3f) +
                               (0.5f + 0.5f * busy) * (0.4f + 0.65f * share * each) * part;
            const float c = rounds * step * (float)(split ? (nk + 3) / 4 + 3 : nk + 3);
            cost = (__float_as_uint(c) & ~63u) + lane;
        }
#pragma unroll
        for (int s = 8; s >= 1; s >>= 1) cost = min(cost, (uint32_t)__shfl_xor((int)cost, s));  // 13 widths at most
        if (lane == 0) {
            plan.cost[wave] = cost >> 6;
            plan.tiles[wave] = tiles;
            plan.width[wave] = kBig - kUnit * (int)(cost & 63u);
        }
    }
    __syncthreads();
    int pick = 3;
#pragma unroll
    for (int i = 2; i >= 0; --i)
        if (plan.cost[i] < plan.cost[pick]) pick = i;
    width = plan.width[pick];
    height = 64 * (pick + 1);
    const int n = plan.tiles[pick];
    number_tiles(plan.t, n_groups, height);
    __syncthreads();
    return n;
}

template <int kForm, typename TO>
__global__ __launch_bounds__(kBigThreads, 1) void gemm_rows_kernel(GemmArgs a) {
    constexpr bool kPc = kForm == kForward;
    constexpr int kStepK = 64;
    __shared__ __attribute__((aligned(1024))) uint8_t p0[32 * 1024];
    __shared__ __attribute__((aligned(1024))) uint8_t p1[32 * 1024];
    __shared__ __attribute__((aligned(1024))) uint8_t q0[32 * 1024];
    __shared__ __attribute__((aligned(1024))) uint8_t q1[32 * 1024];
    __shared__ __attribute__((aligned(1024))) uint8_t x2[16 * 1024];
    __shared__ RowsPlan plan;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int l31 = lane & 31, hi = lane >> 5;
    const int cols = kForm == kForward ? a.N : a.K;  // of the output
    const int n_k = kForm == kForward ? a.K : a.N;   // the contraction, and a row of Q
    const int nk = (n_k + kStepK - 1) / kStepK;
    const size_t w_size = (size_t)a.N * a.K;
    const bool apart = a.p_last != nullptr;
    int width, n_height;
    const int n_tiles = __builtin_amdgcn_readfirstlane(
        plan_rows<kPc ? 16 : 64>(plan, a.offsets, a.n_groups, a.max_rows, cols, nk, width, n_height));
    width = __builtin_amdgcn_readfirstlane(width);
    n_height = __builtin_amdgcn_readfirstlane(n_height);
    const int NB = (cols + width - 1) / width;
    const int n_items = n_tiles * NB;
    const int xcd = blockIdx.x & 7;
    const int per_xcd = gridDim.x >> 3;
    const int i_lo = (int)((long)n_items * xcd / 8);
    const int i_hi = (int)((long)n_items * (xcd + 1) / 8);

    // this lane's fragment offsets in a stage: K-contiguous, of k16 step h; K-strided, of block s
    const int li = lane & 15;
    int offp[4], offq[4];
    if constexpr (kPc) {
        const int r = col_of<TO>(l31);
#pragma unroll
        for (int h = 0; h < 4; ++h) offp[h] = (64 * wn + r) * 128 + ((2 * h + hi) ^ swz_p<TO>(r)) * 16;
    } else {
        const int q = 4 * ((lane >> 4) & 1) + (li & 3), r = 8 * hi + (li >> 2);
#pragma unroll
        for (int s = 0; s < 2; ++s)
            offp[s] = r * 512 + (((2 * wn + s) ^ swz_k(r)) << 6) + col_of<TO>(4 * q) * 2;
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) offq[h] = (32 * wm + l31) * 128 + ((2 * h + hi) ^ swz_q(l31)) * 16;
    // This lane's part of the loads: piece i of a wave is 1 KB of an operand's stage, LDS rows 64 i + 8 wave + [0, 8) of
    // 128 bytes, or 16 i + 2 wave + [0, 2) of 512. Its 16-byte chunk of the row, by the swizzle:
    const int rc = 8 * wave + (lane >> 3), rs = 2 * wave + (lane >> 5);
    const int cp = kPc ? (lane & 7) ^ swz_p<TO>(rc) : (lane & 31) ^ (swz_k(rs) << 2), cq = (lane & 7) ^ swz_q(rc);
    const uint32_t vp = ((uint32_t)(kPc ? rc : rs) * a.K + 8 * cp) * 2, vq = ((uint32_t)rc * n_k + 8 * cq) * 2;
    const uint32_t next_p = (kPc ? 128u : 32u) * a.K, next_q = 128u * n_k;  // bytes from one piece to the next

    // An item by numbers alone; the addresses are made anew from them, as scalars, where they are used (carried
    // through the item loop they would be kept in vector registers, and every load would loop over its lanes).
    struct Item {
        int group, row0, rows, nb;
    };
    struct Tile {
        const uint16_t *p, *q;  // of the first column (forward: its row of w), of the first row
        TO* out;
        int rows, cols, c0;
    };
    auto find = [&](int item) MX_INLINE {
        Item c;
        const MTile t = row_item_at(plan.t, a.n_groups, item, NB, c.nb);
        c.group = t.group;
        c.row0 = t.row0;
        c.rows = t.rows;
        return c;
    };
    auto tile_of = [&](const Item& c) MX_INLINE {
        const int group = __builtin_amdgcn_readfirstlane(c.group), row0 = __builtin_amdgcn_readfirstlane(c.row0);
        Tile t;
        t.rows = __builtin_amdgcn_readfirstlane(c.rows);
        t.c0 = __builtin_amdgcn_readfirstlane(c.nb) * width;
        t.cols = min(width, cols - t.c0);
        t.p = (apart && group == a.n_groups - 1 ? (const uint16_t*)a.p_last : (const uint16_t*)a.p + group * w_size) +
              (kPc ? (size_t)t.c0 * a.K : t.c0);
        t.q = (const uint16_t*)a.q + (size_t)row0 * n_k;
        t.out = (TO*)a.out + (size_t)row0 * cols;
        return t;
    };
    // Piece n of step kc into a stage: P's four, then Q's. What lies outside an operand is not fetched and arrives as
    // zeros: rows past a descriptor's end, and chunks past the contraction or the columns by an offset past every
    // descriptor (a tile's are under 2^26 bytes).
    constexpr uint32_t kPast = 0x40000000u;
    auto piece = [&](const Tile& c, int kc, uint8_t* P, uint8_t* Q, auto n_c) MX_INLINE {
        constexpr int n = decltype(n_c)::value, i = n & 3;
        const uint32_t so = (uint32_t)min(kc, nk - 1) * (kStepK * 2);  // never past the first row's end
        const int left = n_k - kc * kStepK;                            // of the contraction
        if constexpr (n >= 4) {
            lds_buf16(buffer_rsrc(c.q, (uint32_t)c.rows * n_k * 2), vq + i * next_q + (8 * cq < left ? 0u : kPast), so,
                      Q + (8 * i + wave) * 1024);
        } else if constexpr (kPc) {
            lds_buf16(buffer_rsrc(c.p, (uint32_t)c.cols * a.K * 2), vp + i * next_p + (8 * cp < left ? 0u : kPast), so,
                      P + (8 * i + wave) * 1024);
        } else {
            const int rows = max(0, min(kStepK, left));
            lds_buf16(buffer_rsrc(c.p + (size_t)kc * kStepK * a.K, rows ? (uint32_t)(rows * a.K - c.c0) * 2 : 0u),
                      vp + i * next_p + (8 * cp < c.cols ? 0u : kPast), 0, P + (8 * i + wave) * 1024);
        }
    };
    auto load_p = [&](const Tile& c, int kc, uint8_t* P) MX_INLINE {
        piece(c, kc, P, nullptr, std::integral_constant<int, 0>{});
        piece(c, kc, P, nullptr, std::integral_constant<int, 1>{});
        piece(c, kc, P, nullptr, std::integral_constant<int, 2>{});
        piece(c, kc, P, nullptr, std::integral_constant<int, 3>{});
        asm volatile("" ::: "memory");  // in this order: the waits count the loads
    };
    auto load_q = [&](const Tile& c, int kc, uint8_t* Q) MX_INLINE {  // the tile's rows, 64 at a time
        piece(c, kc, nullptr, Q, std::integral_constant<int, 4>{});
        if (c.rows > 64) piece(c, kc, nullptr, Q, std::integral_constant<int, 5>{});
        if (c.rows > 128) piece(c, kc, nullptr, Q, std::integral_constant<int, 6>{});
        if (c.rows > 192) piece(c, kc, nullptr, Q, std::integral_constant<int, 7>{});
        asm volatile("" ::: "memory");
    };
    using C0 = std::integral_constant<int, 0>;
    using C1 = std::integral_constant<int, 1>;
    using C2 = std::integral_constant<int, 2>;
    using C3 = std::integral_constant<int, 3>;
    using C4 = std::integral_constant<int, 4>;
    auto first_loads = [&](const Tile& c) MX_INLINE {
        load_p(c, 0, p0);
        load_q(c, 0, q0);
        load_p(c, 1, p1);
        if (c.rows <= 128) {  // three stages: all but Q of the last
            load_q(c, 1, q0 + 16384);
            load_p(c, 2, q1);
        }
    };
    auto with_nx = [&](int rows, auto f) MX_INLINE {
        if (rows <= 64) f(C1{});
        else if (rows <= 128) f(C2{});
        else if (rows <= 192) f(C3{});
        else f(C4{});
    };

    int item = i_lo + (int)(blockIdx.x >> 3);
    if (item >= i_hi) return;

    // Tiles of 64 x 64, for calls of few tiles, which are as long as their chain of steps: the contraction is split over
    // the four waves of a row half. A step takes 256 of it; the 64 of P's rows (columns, K-strided) that another wave
    // would compute hold the next 64 of the contraction instead, and Q's likewise. (203 rows of 9 groups, 768 x 1280,
    // forward: 13.0 -> 11.1 us; one row of each of 33 groups, 128 x 4096: 26 -> 17.)
    if (width == 64 && n_height == 64) {
        constexpr int kLong = 4 * kStepK;
        const int nl = (n_k + kLong - 1) / kLong;
        for (; item < i_hi; item += per_xcd) {
            const Tile cur = tile_of(find(item));
            auto load = [&](int kc, uint8_t* P, uint8_t* Q) MX_INLINE {
                const int left = n_k - kc * kLong;
                const uint32_t so = (uint32_t)min(kc, nl - 1) * (kLong * 2);
                const __amdgpu_buffer_rsrc_t dq = buffer_rsrc(cur.q, (uint32_t)cur.rows * n_k * 2);
                const int rows = max(0, min(kLong, left));
                const __amdgpu_buffer_rsrc_t dp =
                    kPc ? buffer_rsrc(cur.p, (uint32_t)cur.cols * a.K * 2)
                        : buffer_rsrc(cur.p + (size_t)kc * kLong * a.K, rows ? (uint32_t)(rows * a.K - cur.c0) * 2 : 0u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t v =
                        kPc ? ((uint32_t)rc * a.K + 64 * i + 8 * cp) * 2 + (64 * i + 8 * cp < left ? 0u : kPast)
                            : ((uint32_t)(64 * (cp >> 3) + 16 * i + rs) * a.K + 8 * (cp & 7)) * 2 +
                                  (8 * (cp & 7) < cur.cols ? 0u : kPast);
                    lds_buf16(dp, v, kPc ? so : 0, P + (8 * i + wave) * 1024);
                    lds_buf16(dq, ((uint32_t)rc * n_k + 64 * i + 8 * cq) * 2 + (64 * i + 8 * cq < left ? 0u : kPast), so,
                              Q + (8 * i + wave) * 1024);
                }
                asm volatile("" ::: "memory");  // in this order: the waits count the loads
            };
            f32x16 acc[2] = {};
            auto multiply = [&](const uint8_t* P, const uint8_t* Q) MX_INLINE {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const u32x4 q = *reinterpret_cast<const u32x4*>(Q + wn * 8192 + offq[h]);
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        u32x4 x;
                        if constexpr (kPc) x = *reinterpret_cast<const u32x4*>(P + s * 4096 + offp[h]);
                        else x = lds_read_tr(P + offp[s] + h * 8192);
                        acc[s] = mfma32(x, q, acc[s]);
                    }
                }
            };
            load(0, p0, q0);
            load(1, p1, q1);
            auto step = [&](int kc, uint8_t* P, uint8_t* Q) MX_INLINE {
                wait_vmcnt<8>();  // this step has landed, the next one flies
                mx_barrier();
                multiply(P, Q);
                mx_barrier();  // no wave reads it any more
                load(kc + 2, P, Q);
            };
            for (int kc = 0; kc < nl; kc += 2) {  // a step past the end multiplies zeros
                step(kc, p0, q0);
                step(kc + 1, p1, q1);
            }
            wait_vmcnt<0>();
            mx_barrier();
            // the sums of the four waves, in their order; a register of all lanes is a row of 256 bytes
            float* red = reinterpret_cast<float*>(wave < 4 ? p0 : p1) + (wave & 3) * 2048;
            if (wn > 0) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int r = 0; r < 16; ++r) red[(16 * s + r) * 64 + lane] = acc[s][r];
            }
            mx_barrier();
            if (wn == 0) {
#pragma unroll
                for (int n = 1; n < 4; ++n) {
                    const int from = 2 * n + wm;
                    const float* other = reinterpret_cast<const float*>(from < 4 ? p0 : p1) + (from & 3) * 2048;
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[s][r] += other[(16 * s + r) * 64 + lane];
                }
                const int m = 32 * wm + l31;
                if (m < cur.rows) {
#pragma unroll
                    for (int s = 0; s < 2; ++s)
                        put16(cur.out + (size_t)m * cols + cur.c0, 32 * s, cur.cols, hi, acc[s], a.accumulate != 0);
                }
            }
            mx_barrier();  // the sums are read before the next item's loads
        }
        return;
    }
    Item at = find(item);
    first_loads(tile_of(at));
    for (;;) {
        const bool more = item + per_xcd < i_hi;
        const Tile cur = tile_of(at);
        auto done = [&]() MX_INLINE {
            wait_vmcnt<0>();
            mx_barrier();  // no stage is read or written any more
            if (more) {
                at = find(item + per_xcd);
                first_loads(tile_of(at));
            }
        };
        auto run = [&](auto nx_c) MX_INLINE {
            constexpr int NX = decltype(nx_c)::value;
            // Stages: two of a tile of more than 128 rows, (p0, q0) and (p1, q1); three of a shorter one, whose Q take half
            // the room: (p0, q0), (p1, q0 + 16 KB), (q1, x2)
            constexpr int kStages = NX > 2 ? 2 : 3;
            constexpr int kFly = NX > 2 ? 0 : 4 + NX;  // loads that may be in flight behind the next step's
            f32x16 acc[2][NX] = {};
            u32x4 fp[2][2], fq[2][NX];
            auto read = [&](auto h_c, const uint8_t* P, const uint8_t* Q) MX_INLINE {
                constexpr int h = decltype(h_c)::value, b = h & 1;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if constexpr (kPc) fp[b][s] = *reinterpret_cast<const u32x4*>(P + s * 4096 + offp[h]);
                    else fp[b][s] = lds_read_tr(P + offp[s] + h * 8192);
                }
#pragma unroll
                for (int j = 0; j < NX; ++j) fq[b][j] = *reinterpret_cast<const u32x4*>(Q + j * 8192 + offq[h]);
                __builtin_amdgcn_sched_barrier(0);  // these reads ahead of the products, and no others
            };
            // The products of k16 step h. The loads of a later step stand among those of h = 3 (P) and 0 (Q).
            auto multiply = [&](auto h_c, int kc, uint8_t* P, uint8_t* Q) MX_INLINE {
                constexpr int h = decltype(h_c)::value, b = h & 1;
                auto col = [&](auto j_c) MX_INLINE {
                    constexpr int j = decltype(j_c)::value;
                    if constexpr (j < NX) {
#pragma unroll
                        for (int s = 0; s < 2; ++s) acc[s][j] = mfma32(fp[b][s], fq[b][j], acc[s][j]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if constexpr (h == 3 || (h == 0 && j < NX)) {
                        piece(cur, kc, P, Q, std::integral_constant<int, (h == 3 ? 0 : 4) + j>{});
                        __builtin_amdgcn_sched_barrier(0);
                    }
                };
                col(C0{});
                col(C1{});
                col(C2{});
                col(C3{});
            };
            // A step from stage (P, Q), whose first fragments are in registers; (Pn, Qn) holds the next one, Ql gets the
            // rest of the last.
            auto step = [&](int kc, uint8_t* P, uint8_t* Q, uint8_t* Pn, uint8_t* Qn, uint8_t* Ql) MX_INLINE {
                read(C1{}, P, Q);
                multiply(C0{}, kc + kStages - 1, nullptr, Ql);
                read(C2{}, P, Q);
                multiply(C1{}, 0, nullptr, nullptr);
                read(C3{}, P, Q);
                multiply(C2{}, 0, nullptr, nullptr);
                wait_vmcnt<kFly>();  // the next step has landed
                mx_barrier();        // and no wave reads this stage any more
                read(C0{}, Pn, Qn);
                multiply(C3{}, kc + kStages, P, Q);
            };
            wait_vmcnt<kFly + 4>();
            mx_barrier();
            read(C0{}, p0, q0);
            int kc = 0;  // whole rounds of the ring, then what is left: an exit inside the loop cost 4 to 7%
            if constexpr (kStages == 3) {
                for (; kc + 3 <= nk; kc += 3) {
                    step(kc, p0, q0, p1, q0 + 16384, x2);
                    step(kc + 1, p1, q0 + 16384, q1, x2, q0);
                    step(kc + 2, q1, x2, p0, q0, q0 + 16384);
                }
                if (kc < nk) {
                    step(kc, p0, q0, p1, q0 + 16384, x2);
                    if (kc + 1 < nk) step(kc + 1, p1, q0 + 16384, q1, x2, q0);
                }
            } else {
                for (; kc + 2 <= nk; kc += 2) {
                    step(kc, p0, q0, p1, q1, q1);
                    step(kc + 1, p1, q1, p0, q0, q0);
                }
                if (kc < nk) step(kc, p0, q0, p1, q1, q1);
            }
            done();
#pragma unroll
            for (int j = 0; j < NX; ++j) {
                const int m = 64 * j + 32 * wm + l31;
                if (m >= cur.rows) continue;
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    put16(cur.out + (size_t)m * cols + cur.c0, 64 * wn + 32 * s, cur.cols, hi, acc[s][j],
                          a.accumulate != 0);
            }
        };
        if (64 * wn < cur.cols) {
            with_nx(cur.rows, run);
        } else {  // a wave without columns: its part of the loads
            auto idle = [&](auto nx_c) MX_INLINE {
                constexpr int NX = decltype(nx_c)::value, kStages = NX > 2 ? 2 : 3, kFly = NX > 2 ? 0 : 4 + NX;
                wait_vmcnt<kFly + 4>();
                mx_barrier();
                for (int kc = 0, s = 0; kc < nk; ++kc) {
                    uint8_t* P = s == 0 ? p0 : s == 1 ? p1 : q1;
                    uint8_t* Ql = kStages == 3 ? (s == 0 ? x2 : s == 1 ? q0 : q0 + 16384) : s == 0 ? q1 : q0;
                    load_q(cur, kc + kStages - 1, Ql);
                    wait_vmcnt<kFly>();
                    mx_barrier();
                    load_p(cur, kc + kStages, P);
                    s = s + 1 == kStages ? 0 : s + 1;
                }
            };
            with_nx(cur.rows, idle);
            done();
        }
        if (!more) break;
        item += per_xcd;
    }
}

template <int kForm, typename TO>
moe_status launch_rows(const GemmArgs& a, hipStream_t st) {
    const long cols = kForm == kForward ? a.N : a.K;
    const long tiles = ((long)a.max_rows + 63) / 64 + std::min(a.n_groups, a.max_rows);  // of 64 rows, at most
    const long blocks = (cols + 63) / 64;
    const int grid = (int)std::min((tiles * blocks + 7) / 8 * 8, (long)device_info().cu_count / 8 * 8);
    hipLaunchKernelGGL((gemm_rows_kernel<kForm, TO>), dim3(grid), dim3(kBigThreads), 0, st, a);
    return check_launch("gemm_rows_kernel");
}

// ---------------------------------------------------------------- weights
// dw of a group in tiles of `height` x 256, both operands K-strided, over the group's rows: steps of 32 of them in a ring of
// four stages (steps of 64 in two took 906 us for 8192^3, these 881), since a training batch gives an expert only some
// hundred rows and a ring of short steps ends closer to them. Tiles that short are bound by their stores: 16384 rows
// of 32 experts, 7168 x 2048 in fp32, 654 us, 404 of them without the stores.
template <typename TO>
__global__ __launch_bounds__(kBigThreads, 1) void gemm_weights_kernel(GemmArgs a) {
    constexpr int kStepK = 32;  // rows of a step
    __shared__ __attribute__((aligned(1024))) uint8_t s0[32 * 1024];  // P: 16 KB, Q behind it
    __shared__ __attribute__((aligned(1024))) uint8_t s1[32 * 1024];
    __shared__ __attribute__((aligned(1024))) uint8_t s2[32 * 1024];
    __shared__ __attribute__((aligned(1024))) uint8_t s3[32 * 1024];
    __shared__ int row0[kMaxGroups + 1];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int l31 = lane & 31, hi = lane >> 5;
    const int NB = (a.K + kBig - 1) / kBig, MB = (a.N + a.height - 1) / a.height;
    const size_t w_size = (size_t)a.N * a.K;
    for (int g = threadIdx.x; g <= a.n_groups; g += kBigThreads) row0[g] = clamp_row(a.offsets[g], a.max_rows);
    __syncthreads();
    const int n_items = a.n_groups * MB * NB;
    const int xcd = blockIdx.x & 7;
    const int per_xcd = gridDim.x >> 3;
    const int i_lo = (int)((long)n_items * xcd / 8);
    const int i_hi = (int)((long)n_items * (xcd + 1) / 8);

    // fragments of a stage's block s (P) or j (Q); k16 step h lies 8 KB on
    int offp[2], offq[4];
    {
        const int q = 4 * ((lane >> 4) & 1) + (lane & 3), r = 8 * hi + ((lane & 15) >> 2);
#pragma unroll
        for (int s = 0; s < 2; ++s) offp[s] = r * 512 + (((2 * wn + s) ^ swz_k(r)) << 6) + col_of<TO>(4 * q) * 2;
#pragma unroll
        for (int j = 0; j < 4; ++j) offq[j] = 16384 + r * 512 + (((2 * j + wm) ^ swz_k(r)) << 6) + 8 * q;
    }
    // piece i of a wave is 1 KB of an operand's stage, LDS rows 16 i + 2 wave + [0, 2)
    const int rs = 2 * wave + (lane >> 5), cs = (lane & 31) ^ (swz_k(rs) << 2);
    const uint32_t vp = ((uint32_t)rs * a.K + 8 * cs) * 2, vq = ((uint32_t)rs * a.N + 8 * cs) * 2;

    struct Item {
        int group, mb, nb;
    };
    struct Tile {
        const uint16_t *p, *q;
        TO* out;
        int n_k, c0, o0, rows;  // the group's rows; first column of x and of dy, columns of dy
    };
    auto find = [&](int item) MX_INLINE {
        Item c;
        c.group = item / (MB * NB);
        const int in = item - c.group * (MB * NB);
        c.mb = in / NB;
        c.nb = in - c.mb * NB;
        return c;
    };
    auto tile_of = [&](const Item& c) MX_INLINE {
        const int group = __builtin_amdgcn_readfirstlane(c.group);
        const int r0 = __builtin_amdgcn_readfirstlane(row0[group]), r1 = __builtin_amdgcn_readfirstlane(row0[group + 1]);
        Tile t;
        t.n_k = max(0, r1 - r0);
        t.c0 = __builtin_amdgcn_readfirstlane(c.nb) * kBig;
        t.o0 = __builtin_amdgcn_readfirstlane(c.mb) * a.height;
        t.rows = min(a.height, a.N - t.o0);
        t.p = (const uint16_t*)a.p + (size_t)r0 * a.K;
        t.q = (const uint16_t*)a.q + (size_t)r0 * a.N;
        t.out = (a.out_last && group == a.n_groups - 1 ? (TO*)a.out_last : (TO*)a.out + group * w_size) +
                (size_t)t.o0 * a.K;
        return t;
    };
    // Pieces 2n and 2n + 1 of step kc: P's for n = 0, Q's for n = 1. Rows past the group are not fetched and arrive as
    // zeros; columns past x's row bring the next row's, for outputs that are not kept.
    auto two = [&](const Tile& c, int kc, uint8_t* S, auto n_c) MX_INLINE {
        constexpr bool kQ = decltype(n_c)::value == 1;
        const int ld = kQ ? a.N : a.K, o = kQ ? c.o0 : c.c0;
        const int left = max(0, min(kStepK, c.n_k - kc * kStepK));
        const __amdgpu_buffer_rsrc_t d = buffer_rsrc((kQ ? c.q : c.p) + (size_t)kc * kStepK * ld + o,
                                                     left ? (uint32_t)(left * ld - o) * 2 : 0u);
        uint8_t* l = S + (kQ ? 16384 : 0) + wave * 1024;
        const uint32_t v = kQ ? vq + (8 * cs < c.rows ? 0u : 0x40000000u) : vp;
        lds_buf16(d, v, 0, l);
        __builtin_amdgcn_sched_barrier(0);
        return [=]() MX_INLINE { lds_buf16(d, v + 32u * ld, 0, l + 8192); };
    };
    using C0 = std::integral_constant<int, 0>;
    using C1 = std::integral_constant<int, 1>;
    using C2 = std::integral_constant<int, 2>;
    using C3 = std::integral_constant<int, 3>;
    using C4 = std::integral_constant<int, 4>;
    auto whole = [&](const Tile& c, int kc, uint8_t* S) MX_INLINE {
        two(c, kc, S, C0{})();
        two(c, kc, S, C1{})();
        asm volatile("" ::: "memory");  // in this order: the waits count the loads
    };
    auto first_loads = [&](const Tile& c) MX_INLINE {
        whole(c, 0, s0);
        whole(c, 1, s1);
        whole(c, 2, s2);
        two(c, 3, s3, C0{})();
        asm volatile("" ::: "memory");
    };
    auto with_nx = [&](int rows, auto f) MX_INLINE {
        if (rows <= 64) f(C1{});
        else if (rows <= 128) f(C2{});
        else if (rows <= 192) f(C3{});
        else f(C4{});
    };

    int item = i_lo + (int)(blockIdx.x >> 3);
    if (item >= i_hi) return;
    Item at = find(item);
    first_loads(tile_of(at));
    for (;;) {
        const bool more = item + per_xcd < i_hi;
        const Tile cur = tile_of(at);
        if (more) at = find(item + per_xcd);
        auto run = [&](auto nx_c) MX_INLINE {
            constexpr int NX = decltype(nx_c)::value;
            const int nk = (cur.n_k + kStepK - 1) / kStepK;
            f32x16 acc[2][NX] = {};
            u32x4 fp[2][2], fq[2][NX];
            auto read = [&](auto h_c, const uint8_t* S) MX_INLINE {
                constexpr int h = decltype(h_c)::value;
#pragma unroll
                for (int s = 0; s < 2; ++s) fp[h][s] = lds_read_tr(S + offp[s] + h * 8192);
#pragma unroll
                for (int j = 0; j < NX; ++j) fq[h][j] = lds_read_tr(S + offq[j] + h * 8192);
                __builtin_amdgcn_sched_barrier(0);  // these reads ahead of the products, and no others
            };
            // the products of k16 step h, half of a later step's loads among them
            auto multiply = [&](auto h_c, int kc, uint8_t* S) MX_INLINE {
                constexpr int h = decltype(h_c)::value;
                auto col = [&](auto j_c) MX_INLINE {
                    constexpr int j = decltype(j_c)::value;
                    if constexpr (j < NX) {
#pragma unroll
                        for (int s = 0; s < 2; ++s) acc[s][j] = sizeof(TO) == 4 ? mfma32(fq[h][j], fp[h][s], acc[s][j]) : mfma32(fp[h][s], fq[h][j], acc[s][j]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                };
                col(C0{});
                auto second = two(cur, kc, S, std::integral_constant<int, 1 - h>{});
                col(C1{});
                col(C2{});
                second();
                __builtin_amdgcn_sched_barrier(0);
                col(C3{});
            };
            // A step from stage S, whose first fragments are in registers; Sn holds the next one, Sp is the one before,
            // of which P is loaded.
            auto step = [&](int kc, uint8_t* S, uint8_t* Sn, uint8_t* Sp) MX_INLINE {
                read(C1{}, S);
                multiply(C0{}, kc + 3, Sp);
                wait_vmcnt<8>();  // the next step has landed, two fly
                mx_barrier();     // and no wave reads this stage any more
                read(C0{}, Sn);
                multiply(C1{}, kc + 4, S);
            };
            wait_vmcnt<10>();
            mx_barrier();
            read(C0{}, s0);
            int kc = 0;
            for (; kc + 4 <= nk; kc += 4) {
                step(kc, s0, s1, s3);
                step(kc + 1, s1, s2, s0);
                step(kc + 2, s2, s3, s1);
                step(kc + 3, s3, s0, s2);
            }
            if (kc < nk) {
                step(kc, s0, s1, s3);
                if (kc + 1 < nk) {
                    step(kc + 1, s1, s2, s0);
                    if (kc + 2 < nk) step(kc + 2, s2, s3, s1);
                }
            }
            wait_vmcnt<0>();
            mx_barrier();  // no stage is read or written any more
            // The next item's loads go ahead of the stores, but behind fp32 ones (854 -> 740 us by that and by whole lines,
            // 767 by lines alone; bf16 1148 us, 1179 behind).
            if (more && sizeof(TO) == 2) first_loads(tile_of(at));
            if (nk > 0 || !a.accumulate) {
                if constexpr (sizeof(TO) == 4) {
                    const __amdgpu_buffer_rsrc_t d = buffer_rsrc(cur.out, (uint32_t)cur.rows * a.K * 4);
                    uint32_t v[2];
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int c = cur.c0 + 64 * wn + 32 * s + l31;
                        v[s] = c < a.K ? ((uint32_t)(32 * wm + 4 * hi) * a.K + c) * 4 : 0x40000000u;
                    }
                    auto put = [&](auto add_c) MX_INLINE {
#pragma unroll
                        for (int j = 0; j < NX; ++j)
#pragma unroll
                            for (int r = 0; r < 16; ++r)
#pragma unroll
                                for (int s = 0; s < 2; ++s) {
                                    const uint32_t at = v[s] + (uint32_t)(64 * j + 8 * (r / 4) + r % 4) * a.K * 4;
                                    float x = acc[s][j][r];
                                    if constexpr (decltype(add_c)::value)
                                        x += __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(d, at, 0, 0));
                                    // not kept in L2, where 256 CUs' tiles push out the operands: 743 -> 669 us
                                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), d, at, 0, kNonTemporal);
                                }
                    };
                    if (a.accumulate) put(std::true_type{});
                    else put(std::false_type{});
                } else if (!a.accumulate) {
                    const __amdgpu_buffer_rsrc_t d = buffer_rsrc(cur.out, (uint32_t)cur.rows * a.K * 2);
#pragma unroll
                    for (int j = 0; j < NX; ++j)
                        put_block(d, a.K, 64 * j + 32 * wm, cur.c0 + 64 * wn, a.K, lane, acc[0][j], acc[1][j]);
                } else
#pragma unroll
                for (int j = 0; j < NX; ++j) {
                    const int m = 64 * j + 32 * wm + l31;
                    if (m >= cur.rows) continue;
#pragma unroll
                    for (int s = 0; s < 2; ++s)
                        put16(cur.out + (size_t)m * a.K, cur.c0 + 64 * wn + 32 * s, a.K, hi, acc[s][j],
                              a.accumulate != 0);
                }
            }
        };
        with_nx(cur.rows, run);
        if (!more) break;
        if (sizeof(TO) == 4) first_loads(tile_of(at));
        item += per_xcd;
    }
}

// The height with the shortest estimate: the rounds of items that a workgroup walks, times a tile's stores (0.049 h us in
// bf16, 1.6 times that in fp32) and its steps (0.3 + 0.0011 h us each), at the bound's rows for each group. 5000 rows of
// one group, 256 x 7168: 93 us in tiles of 256 rows, 48 of 64; 16384 of 32, 7168 x 2048: 562 of 256, 1173 of 64; 150 of 16, 680 x
// 680: 8.4 and 10.2, 7.9 of 192.
template <typename TO>
moe_status launch_weights(GemmArgs a, hipStream_t st) {
    const int grid_max = device_info().cu_count / 8 * 8;
    const float steps = (float)a.max_rows / (float)a.n_groups / 32.0f + 1.0f;
    const long blocks = (long)a.n_groups * ((a.K + kBig - 1) / kBig);
    long items = 0;
    float best = 0.f;
    for (int h = kBig; h >= 64; h -= 64) {
        const long n = blocks * ((a.N + h - 1) / h);
        const float rounds = (float)((n + grid_max - 1) / grid_max);
        const float cost = rounds * (0.049f * h * (sizeof(TO) == 4 ? 1.6f : 1.0f) + steps * (0.3f + 0.0011f * h));
        if (h == kBig || cost < best) {
            best = cost;
            items = n;
            a.height = h;
        }
    }
    const int grid = (int)std::min((items + 7) / 8 * 8, (long)grid_max);
    hipLaunchKernelGGL(gemm_weights_kernel<TO>, dim3(grid), dim3(kBigThreads), 0, st, a);
    return check_launch("gemm_weights_kernel");
}

template <int kForm>
moe_status launch_form(const GemmArgs& a, moe_dtype dt, moe_dtype out_dt, hipStream_t st) {
    if (dt == MOE_F32) return launch_f32<kForm>(a, st);
    if constexpr (kForm == kWeights)
        return out_dt == MOE_F32 ? launch_weights<float>(a, st) : launch_weights<uint16_t>(a, st);
    else
        return out_dt == MOE_F32 ? launch_rows<kForm, float>(a, st) : launch_rows<kForm, uint16_t>(a, st);
}

}  // namespace

moe_status launch_grouped_gemm(const void* x, const void* w, const void* w_last, moe_dtype dt, const int32_t* offsets,
                               int n_groups, int max_rows, int N, int K, void* y, moe_dtype y_dt, int accumulate,
                               hipStream_t st) {
    return launch_form<kForward>(GemmArgs{w, w_last, x, offsets, n_groups, max_rows, N, K, y, nullptr, accumulate}, dt,
                                 y_dt, st);
}
moe_status launch_grouped_gemm_dx(const void* dy, const void* w, const void* w_last, moe_dtype dt,
                                  const int32_t* offsets, int n_groups, int max_rows, int N, int K, void* dx,
                                  moe_dtype dx_dt, int accumulate, hipStream_t st) {
    return launch_form<kInput>(GemmArgs{w, w_last, dy, offsets, n_groups, max_rows, N, K, dx, nullptr, accumulate}, dt,
                               dx_dt, st);
}
moe_status launch_grouped_gemm_dw(const void* dy, const void* x, moe_dtype dt, const int32_t* offsets, int n_groups,
                                  int max_rows, int N, int K, void* dw, void* dw_last, moe_dtype dw_dt, int accumulate,
                                  hipStream_t st) {
    return launch_form<kWeights>(GemmArgs{x, nullptr, dy, offsets, n_groups, max_rows, N, K, dw, dw_last, accumulate},
                                 dt, dw_dt, st);
}

}  // namespace moe
