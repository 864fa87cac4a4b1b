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
#include "ffn_dev.h"

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
};

// ============================================================================ tiles of 128 x 128
// 4 waves of 64 x 64, operands through registers into LDS, two stages. One
// step takes 64 bytes of the contraction from each K-contiguous row, or 32
// (fp32: 16) rows of 128 columns of a K-strided operand.
constexpr int kT = 128;
constexpr int kStepBytes = 64;

template <typename T>
struct Step {
    static constexpr int k = kStepBytes / sizeof(T);
    static constexpr int vec = 16 / sizeof(T);                 // elements of a 16-byte piece
    static constexpr int kc_row = kStepBytes + 16;             // LDS bytes of a K-contiguous row
    static constexpr int ks_row = kT * (int)sizeof(T) + 16;    // and of a K-strided one
    static constexpr int bytes = kT * kc_row > k * ks_row ? kT * kc_row : k * ks_row;
};

// this thread's two 16-byte pieces of a step's operand tile; what lies outside the operand is zero
template <typename T, bool kContig>
__device__ __forceinline__ void fetch(const T* base, size_t ld, int n_out, int out0, int n_k, int k0, u32x4* r) {
    using S = Step<T>;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int piece = threadIdx.x + 256 * i;
        int o, k;
        if constexpr (kContig) {
            o = out0 + (piece >> 2);
            k = k0 + (piece & 3) * S::vec;
        } else {
            constexpr int per_row = kT / S::vec;
            k = k0 + piece / per_row;
            o = out0 + piece % per_row * S::vec;
        }
        r[i] = u32x4{0, 0, 0, 0};
        if (o < n_out && k < n_k)
            r[i] = *reinterpret_cast<const u32x4*>(base + (kContig ? (size_t)o * ld + k : (size_t)k * ld + o));
    }
}
template <typename T, bool kContig>
__device__ __forceinline__ void stage(uint8_t* l, const u32x4* r) {
    using S = Step<T>;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int piece = threadIdx.x + 256 * i;
        constexpr int per_row = kT / S::vec;
        const int at = kContig ? (piece >> 2) * S::kc_row + (piece & 3) * 16
                               : piece / per_row * S::ks_row + piece % per_row * 16;
        *reinterpret_cast<u32x4*>(l + at) = r[i];
    }
}
// lane (li, lk) of a 16-wide block at output o0: its 16 bytes of the contraction, elements lk * vec + [0, vec)
template <typename T, bool kContig>
__device__ __forceinline__ u32x4 fragment(const uint8_t* l, int o0, int li, int lk) {
    using S = Step<T>;
    if constexpr (kContig) {
        return *reinterpret_cast<const u32x4*>(l + (o0 + li) * S::kc_row + lk * 16);
    } else {
        union {
            T e[S::vec];
            u32x4 v;
        } u;
#pragma unroll
        for (int j = 0; j < S::vec; ++j)
            u.e[j] = *reinterpret_cast<const T*>(l + (lk * S::vec + j) * S::ks_row + (o0 + li) * sizeof(T));
        return u.v;
    }
}
__device__ __forceinline__ f32x4 mfma_step(u32x4 a, u32x4 b, f32x4 c, uint16_t) { return mfma_bf16(a, b, c); }
__device__ __forceinline__ f32x4 mfma_step(u32x4 a, u32x4 b, f32x4 c, float) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[t]), __uint_as_float(b[t]), c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ void put4(uint16_t* o, f32x4 v, bool add) {
    uint2* p = reinterpret_cast<uint2*>(o);
    if (add) {
        const uint2 old = *p;
        v += f32x4{bf16_lo(old.x), bf16_hi(old.x), bf16_lo(old.y), bf16_hi(old.y)};
    }
    *p = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void put4(float* o, f32x4 v, bool add) {
    f32x4* p = reinterpret_cast<f32x4*>(o);
    if (add) v += *p;
    *p = v;
}

template <typename T, typename TO, int kForm>
__global__ __launch_bounds__(256) void gemm_tile_kernel(GemmArgs a) {
    using S = Step<T>;
    constexpr bool kPc = kForm == kForward, kQc = kForm != kWeights;
    __shared__ __attribute__((aligned(16))) uint8_t lp[2][S::bytes], lq[2][S::bytes];
    __shared__ TileMap tm;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, lk = lane >> 4;
    const int cols = kForm == kForward ? a.N : a.K;  // of the output
    const int NB = (cols + kT - 1) / kT, MB = (a.N + kT - 1) / kT;
    const size_t w_size = (size_t)a.N * a.K;
    const bool apart = kForm == kWeights ? a.out_last != nullptr : a.p_last != nullptr;
    int n_items;
    if constexpr (kForm == kWeights) n_items = a.n_groups * MB * NB;
    else n_items = build_tile_map(tm, a.offsets, a.n_groups, a.max_rows, kT) * NB;

    for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
        const T *p, *q;
        TO* out;
        int nb, q0, rows, n_k;  // column block; first output row, rows that end the tile, length of the contraction
        if constexpr (kForm == kWeights) {
            const int g = item / (MB * NB), in = item % (MB * NB);
            const int r0 = clamp_row(a.offsets[g], a.max_rows), r1 = clamp_row(a.offsets[g + 1], a.max_rows);
            nb = in % NB;
            q0 = in / NB * kT;
            rows = a.N;
            n_k = max(0, r1 - r0);
            p = (const T*)a.p + (size_t)r0 * a.K;
            q = (const T*)a.q + (size_t)r0 * a.N;
            out = apart && g == a.n_groups - 1 ? (TO*)a.out_last : (TO*)a.out + g * w_size;
        } else {
            const MTile t = item_at(tm, a.offsets, a.n_groups, a.max_rows, item, NB, kT, nb);
            n_k = kForm == kForward ? a.K : a.N;
            p = apart && t.group == a.n_groups - 1 ? (const T*)a.p_last : (const T*)a.p + t.group * w_size;
            q = (const T*)a.q + (size_t)t.row0 * n_k;
            out = (TO*)a.out + (size_t)t.row0 * cols;
            q0 = 0;
            rows = t.rows;
        }
        const size_t ldq = kForm == kForward ? a.K : a.N;
        f32x4 acc[4][4] = {};
        u32x4 rp[2], rq[2];
        const int nk = (n_k + S::k - 1) / S::k;
        auto load = [&](int kc) {
            fetch<T, kPc>(p, a.K, cols, nb * kT, n_k, kc * S::k, rp);
            fetch<T, kQc>(q, ldq, rows, q0, n_k, kc * S::k, rq);
        };
        __syncthreads();  // the previous item's reads
        if (nk > 0) {
            load(0);
            stage<T, kPc>(lp[0], rp);
            stage<T, kQc>(lq[0], rq);
        }
        for (int kc = 0; kc < nk; ++kc) {
            __syncthreads();
            if (kc + 1 < nk) load(kc + 1);
            u32x4 fp[4], fq[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                fp[i] = fragment<T, kPc>(lp[kc & 1], 64 * (wave & 1) + 16 * i, li, lk);
                fq[i] = fragment<T, kQc>(lq[kc & 1], 64 * (wave >> 1) + 16 * i, li, lk);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = mfma_step(fp[i], fq[j], acc[i][j], T{});
            if (kc + 1 < nk) {  // the other stage: its readers passed this step's barrier
                stage<T, kPc>(lp[(kc + 1) & 1], rp);
                stage<T, kQc>(lq[(kc + 1) & 1], rq);
            }
        }
        // lane (li, lk): columns 4 lk + [0, 4) of the block at output row li
        if (kForm == kWeights && nk == 0 && a.accumulate) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = q0 + 64 * (wave >> 1) + 16 * j + li;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = nb * kT + 64 * (wave & 1) + 16 * i + 4 * lk;
                if (r < rows && c < cols) put4(out + (size_t)r * cols + c, acc[i][j], a.accumulate != 0);
            }
        }
    }
}

template <typename T, typename TO, int kForm>
moe_status launch_tiles(const GemmArgs& a, hipStream_t st) {
    const long nb = ((kForm == kForward ? a.N : a.K) + kT - 1) / kT;
    const long tiles = kForm == kWeights ? (long)a.n_groups * ((a.N + kT - 1) / kT)
                                         : ((long)a.max_rows + kT - 1) / kT + std::min(a.n_groups, a.max_rows);
    const int grid = (int)std::min(tiles * nb, (long)device_info().cu_count * 2);
    hipLaunchKernelGGL((gemm_tile_kernel<T, TO, kForm>), dim3(grid), dim3(256), 0, st, a);
    return check_launch("gemm_tile_kernel");
}

template <int kForm>
moe_status launch_form(const GemmArgs& a, moe_dtype dt, moe_dtype out_dt, hipStream_t st) {
    if (dt == MOE_F32) return launch_tiles<float, float, kForm>(a, st);
    if (out_dt == MOE_F32) return launch_tiles<uint16_t, float, kForm>(a, st);
    return launch_tiles<uint16_t, uint16_t, kForm>(a, st);
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
