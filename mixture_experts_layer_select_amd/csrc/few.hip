// The whole MoE layer for a few tokens with MXFP4 experts. At most 16 tokens
// are the columns of one 16x16x128 MFMA, so every hit expert's weights cross
// HBM once whatever the number of tokens that picked it, and an expert's
// product is taken for all 16 columns at no extra cost; only picked
// (token, expert) pairs are kept. Bound by HBM: 3 H I (1/2 + 1/32) bytes per
// distinct hit expert. Three kernels:
//
//   logits: one wave per (token, expert), the same bits as moe_route's.
//   gate/up: every workgroup picks the experts from the logits itself (one wave
//     per token), which costs less than a kernel of its own. An item is 8 to 32
//     intermediate columns of one expert (8 gate and 8 up rows, one MFMA
//     operand, to a wave); 8 to 2 waves split K, by its length, and add their
//     partial sums through LDS. Items are I/8 to I/32 per hit expert, so with
//     one workgroup per CU the load is even for any number of experts. The
//     quantised tokens stay in registers for the whole kernel. Items of the
//     shared expert come first: the load of the first one does not wait for the
//     routing.
//   down + combine: a workgroup owns up to 32 columns of the output for every
//     hit expert; the waves split K (and the experts, where K is short) and add
//     each expert's product, times its routing weight, in fp32 registers until
//     the end. One rounding, no
//     atomics, and a token's sum depends neither on the schedule nor on the
//     other tokens. The intermediate is quantised into LDS, as many
//     (expert, token) rows at a time as fit.
//
// Both products stream the weights from HBM into LDS with direct loads, each
// wave for itself: 8 rows of 128 bytes per load, the next item's or the next
// two units' loads in flight while one is multiplied, so no wave waits for
// another's data. Weights read straight into the MFMA's registers (16 rows of
// 64 bytes per load, waited for before each product) reached 2.7 and 2.0 TB/s.
// At H = 7168, I = 2048 one token's nine experts take 29 + 17 us behind 4.7 of
// logits (140 and 70 MB; 6 TB/s once the weights run, 2 to 5 us after the start),
// eight tokens' 58 take 150 to 166 + 87 to 95 us (5.4 TB/s in all).
#include "mx_dev.h"
#include "route_dev.h"

namespace moe {
namespace {

constexpr int kFewT = 16;      // tokens: the columns of one MFMA
constexpr int kFewK = 8;       // picks per token
constexpr int kFewSlots = kFewT * kFewK;
constexpr int kFewGroups = kFewSlots + 1;
constexpr int kFewMaxE = 512;  // local experts: checked by the C entry
constexpr int kFewThreads = 512;
constexpr int kFewWaves = kFewThreads / 64;
constexpr int kFewPairs = 4;   // K steps of 256 per wave of the gate/up kernel, at most: H <= 8192

struct FewArgs {
    const uint16_t* x;         // [T][H] bf16
    const float* logits;       // [T][E], or null: ids and weights are given
    int32_t* ids;              // [T][k]
    float* topk_w;             // [T][k]
    int T, k, E, scoring, renorm, H, I, base, E_local, has_shared;
    const uint8_t *w13, *w13s, *w2, *w2s, *ws13, *ws13s, *ws2, *ws2s;
    struct FewGroups* groups;  // the map, from the gate/up kernel to the down kernel
    float* a;                  // [T*k + T][I] fp32 intermediate, row = slot (T*k + t: shared)
    uint16_t* out;             // [T][H] bf16
    int cols;                  // output columns per workgroup of the down kernel
};

// The groups: the shared expert (if any), then the distinct local experts among
// the picks, ascending. The gate/up kernel's workgroups build it; the first one
// leaves it in memory for the down kernel, which so knows its experts one load
// after its start.
struct FewGroups {
    int n;
    int expert[kFewGroups];              // -1: the shared one
    uint32_t mask[kFewGroups];           // the tokens that picked it
    short slot[kFewGroups * kFewT + 2];  // the first slot of a token that did, -1: none
};
static_assert(sizeof(FewGroups) % 4 == 0, "copied by dwords");
struct FewMap {
    __attribute__((aligned(16))) uint32_t hit[kFewMaxE / 32];  // the local experts among the picks
    int id[kFewSlots + kFewK];           // local expert of a slot, -1: none
    float w[kFewSlots + kFewK];
    FewGroups g;
};
// ... and what the down kernel makes of it
struct FewSum {
    int id[kFewSlots + kFewK];
    float w[kFewSlots + kFewK];
    float weight[kFewGroups * kFewT];    // the sum of a token's weights (an id may stand twice in a row)
    int pre[kFewGroups + 1];             // picked (group, token) pairs before each group
    short pair_slot[kFewSlots + kFewT];  // the pairs in order: slot and group
    short pair_group[kFewSlots + kFewT];
};

__device__ __forceinline__ int few_local(const FewArgs& p, int id) {  // any value: no overflow
    return id >= p.base && id - p.base < p.E_local ? id - p.base : -1;
}

// Before the barrier behind which m.id (-1 behind the T k slots) is seen
__device__ __forceinline__ void init_few_map(FewMap& m, const FewArgs& p) {
    const int tid = threadIdx.x, S = p.T * p.k;
    if (tid < kFewMaxE / 32) m.hit[tid] = 0;
    for (int i = tid; i < kFewGroups * kFewT; i += kFewThreads)
        m.g.slot[i] = (short)(p.has_shared && i < p.T ? S + i : -1);
    for (int i = tid; i < kFewGroups; i += kFewThreads) m.g.mask[i] = p.has_shared && i == 0 ? (1u << p.T) - 1 : 0;
}

// Builds the map behind that barrier and returns the number of groups. All
// threads call; ends with a barrier.
__device__ __forceinline__ int build_few_map(FewMap& m, const FewArgs& p) {
    const int tid = threadIdx.x, sh = p.has_shared ? 1 : 0;
    const int e = tid < kFewSlots ? m.id[tid] : -1;
    if (e >= 0) atomicOr(&m.hit[e >> 5], 1u << (e & 31));
    mx_barrier();
    int n = sh, rank = sh;  // an expert's rank: the hit ones below it
#pragma unroll
    for (int w = 0; w < kFewMaxE / 32; ++w) {
        const uint32_t hit = m.hit[w];
        const int below = min(max(e - 32 * w, 0), 32);
        rank += __popc(below < 32 ? hit & ((1u << below) - 1) : hit);
        n += __popc(hit);
    }
    if (tid == 0) {
        m.g.n = n;
        if (sh) m.g.expert[0] = -1;
    }
    if (e >= 0) {
        const int t = tid / p.k, j0 = tid - t * p.k;
        bool first = true;  // of its token's picks
#pragma unroll
        for (int j = 0; j < kFewK; ++j)
            if (j < j0 && m.id[tid - j0 + j] == e) first = false;
        m.g.expert[rank] = e;
        if (first) {
            m.g.slot[rank * kFewT + t] = (short)tid;
            atomicOr(&m.g.mask[rank], 1u << t);
        }
    }
    mx_barrier();
    return __builtin_amdgcn_readfirstlane(n);
}

// Behind a barrier that shows g, s.id and s.w; ends with one
__device__ __forceinline__ void sum_few_map(const FewGroups& g, FewSum& s, int n, const FewArgs& p) {
    const int tid = threadIdx.x, sh = p.has_shared ? 1 : 0;
    if (tid < 64) {
        int run = 0;
        for (int g0 = 0; g0 < n; g0 += 64) {
            const int c = g0 + tid < n ? __popc(g.mask[g0 + tid]) : 0;
            int sum = c;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(sum, d);
                if (tid >= d) sum += o;
            }
            if (g0 + tid < n) s.pre[g0 + tid] = run + sum - c;
            run += __shfl(sum, 63);
        }
        if (tid == 0) s.pre[n] = run;
    }
    for (int i = tid; i < n * kFewT; i += kFewThreads) {
        const int gr = i / kFewT, t = i % kFewT;
        float w = gr < sh ? 1.0f : 0.f;
        if (gr >= sh && g.mask[gr] >> t & 1) {
            const int id = s.id[g.slot[i]];
#pragma unroll
            for (int j = kFewK - 1; j >= 0; --j)
                if (j < p.k && s.id[t * p.k + j] == id) w += s.w[t * p.k + j];
        }
        s.weight[i] = w;
    }
    mx_barrier();
    for (int i = tid; i < n * kFewT; i += kFewThreads) {
        const int gr = i / kFewT, t = i % kFewT;
        const uint32_t mask = g.mask[gr];
        if (mask >> t & 1) {
            const int at = s.pre[gr] + __popc(mask & ((1u << t) - 1));
            s.pair_slot[at] = g.slot[i];
            s.pair_group[at] = (short)gr;
        }
    }
    mx_barrier();
}

__device__ __forceinline__ f32x4 mfma16_fp4(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
    const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// LDS rows of 128 bytes: chunk c (16 bytes) of row r sits at chunk c ^ (r & 7),
// so the 16 rows of one MFMA operand spread over the banks
__device__ __forceinline__ uint32_t few_at(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// A byte offset of which the compiler knows nothing. A direct load to LDS
// counts as a store of one lane's bytes at its first address; a read that is
// proven apart from every such store is made to wait for all loads in flight.
__device__ __forceinline__ uint32_t few_opaque(uint32_t v) {
    asm("" : "+v"(v));
    return v;
}

// ---------------------------------------------------------------- gate/up
constexpr int kGuCodes = 16 * 128 * kFewPairs;  // a wave's share of one item
constexpr int kGuStage = kGuCodes + 16 * 8 * kFewPairs;  // ... and its scales
constexpr int kGuLoads = 2 * kFewPairs + 2;     // its loads: codes, and two for the scales

// ks: waves that share an item's K, 2, 4 or 8
template <int ks>
__global__ __launch_bounds__(kFewThreads) void few_gate_up_kernel(FewArgs p) {
    // a stage is an object of its own, so that reads of one do not wait for loads into the other
    __shared__ __attribute__((aligned(1024))) uint8_t s0[kFewWaves][kGuStage];
    __shared__ __attribute__((aligned(1024))) uint8_t s1[kFewWaves][kGuStage];
    __shared__ __attribute__((aligned(16))) float red[2][kFewWaves][kFewT][16];
    __shared__ FewMap m;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, lk = lane >> 4;
    const int rowb = p.H / 2, kb = p.H / kMxBlock;
    // the wave's slice of K and its 8 columns of the item
    constexpr int width = 8 * kFewWaves / ks;
    const int ksi = wave & (ks - 1), cg = wave / ks;
    const int np = p.H / 256, p0 = ksi * np / ks, cnt = (ksi + 1) * np / ks - p0;
    const int S = p.T * p.k, sh = p.has_shared ? 1 : 0;
    const int per = p.I / width, G = gridDim.x;

    // a load: the 8 gate or the 8 up rows of an item for one K step
    const uint32_t wv = (uint32_t)((8 * cg + (lane >> 3)) * rowb + p0 * 128 + (((lane & 7) ^ (lane >> 3)) << 4));
    const uint32_t up = (uint32_t)p.I * rowb;
    const uint32_t sv = (uint32_t)((8 * cg + (lane >> 3)) * kb + p0 * 8 + (lane & 7) * 4), sup = (uint32_t)p.I * kb;
    auto issue = [&](int it, int n, uint8_t (&st)[kFewWaves][kGuStage]) MX_INLINE {
        const bool on = it < n * per;  // items past the end load nothing, but count
        const int g = on ? it / per : 0, i0 = on ? it % per * width : 0;
        const int e = on && g >= sh ? __builtin_amdgcn_readfirstlane(m.g.expert[g]) : 0;
        const size_t rows = 2 * (size_t)p.I;
        const uint8_t* W = (g < sh ? p.ws13 : p.w13 + e * rows * rowb) + (size_t)i0 * rowb;
        const uint8_t* Ws = (g < sh ? p.ws13s : p.w13s + e * rows * kb) + (size_t)i0 * kb;
        const uint32_t left = (uint32_t)(rows - i0), c = on ? cnt : 0;  // K steps past this wave's neither
        const __amdgpu_buffer_rsrc_t sd = buffer_rsrc(Ws, on ? left * kb : 0);
        lds_buf4(sd, sv, 0, st[wave] + kGuCodes);
        lds_buf4(sd, sv, sup, st[wave] + kGuCodes + 256);
#pragma unroll
        for (uint32_t j = 0; j < kFewPairs; ++j) {
            const __amdgpu_buffer_rsrc_t wd = buffer_rsrc(W, j < c ? left * rowb : 0);
            lds_buf16(wd, wv, j * 128, st[wave] + j * 2048);
            lds_buf16(wd, wv, j * 128 + up, st[wave] + j * 2048 + 1024);
        }
        asm volatile("" ::: "memory");  // loads of different stages stay in order: the waits count them
    };

    int it = blockIdx.x;
    // an item of the shared expert needs no routing; a wave that picks experts waits for its logits alone first
    const bool early = it < sh * per && !(p.logits && wave < p.T);
    if (early) issue(it, 1, s0);
    if (p.logits)
        for (int t = wave; t < p.T; t += kFewWaves)
            route_topk_token<1>(p.logits, p.T, p.E, p.k, p.scoring, p.renorm, m.id, m.w, t);
    // The tokens, quantised as moe_quantize_mxfp4 does, eight values per thread, into the stage that is filled last:
    // codes, then scales. (A lane that reads a block of its own costs the address unit a line per lane: four times
    // the time.)
    uint8_t* const xq = &s1[0][0];
    const int blocks = p.T * kb;
    static_assert(kFewT * kFewPairs * kFewWaves * 256 / kMxBlock * 17 <= sizeof(s1), "the tokens fit the stage");
    const __amdgpu_buffer_rsrc_t xd = buffer_rsrc(p.x, (uint32_t)(p.T * p.H * 2));
    constexpr int kBatch = 4;
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < 4 * blocks; i0 += kBatch * kFewThreads) {
        u32x4 raw[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) raw[q] = buffer_load16(xd, (uint32_t)(i0 + q * kFewThreads) * 16, 0);
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int i = i0 + q * kFewThreads;
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = bf16_lo(raw[q][j]);
                v[2 * j + 1] = bf16_hi(raw[q][j]);
            }
            uint32_t byte;
            const uint32_t code = mx_quantise8(v, byte);
            if (i < 4 * blocks) {
                *reinterpret_cast<uint32_t*>(xq + i * 4) = code;
                if ((i & 3) == 0) xq[blocks * 16 + (i >> 2)] = (uint8_t)byte;
            }
        }
    }
    init_few_map(m, p);
    if (!p.logits && threadIdx.x < kFewSlots)
        m.id[threadIdx.x] = threadIdx.x < S ? few_local(p, p.ids[threadIdx.x]) : -1;
    mx_barrier();
    // lane (li, lk) holds token li's block lk of each of its wave's half steps; columns past T repeat the last token
    u32x4 b[2 * kFewPairs];
    uint32_t sb[2 * kFewPairs];
#pragma unroll
    for (int q = 0; q < 2 * kFewPairs; ++q) {
        const int at = min(li, p.T - 1) * kb + min(2 * p0 + q, 2 * np - 1) * 4 + lk;
        b[q] = *reinterpret_cast<const u32x4*>(xq + at * 16);
        sb[q] = xq[blocks * 16 + at] & (q < 2 * cnt ? 0xffu : 0u);
    }
    if (p.logits && threadIdx.x < kFewSlots) {
        const int id = threadIdx.x < S ? m.id[threadIdx.x] : -1;
        if (blockIdx.x == 0 && threadIdx.x < S) {
            p.ids[threadIdx.x] = id;
            p.topk_w[threadIdx.x] = m.w[threadIdx.x];
        }
        m.id[threadIdx.x] = threadIdx.x < S ? few_local(p, id) : -1;
    }
    mx_barrier();
    const int n = build_few_map(m, p);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < (int)(sizeof(FewGroups) / 4); i += kFewThreads)
            reinterpret_cast<uint32_t*>(p.groups)[i] = reinterpret_cast<const uint32_t*>(&m.g)[i];
    if (!early) issue(it, n, s0);
    wait_vmcnt<0>();  // said once here, or the compiler says it in the loop, before the first stage's reads
    issue(it + G, n, s1);

    const uint32_t srow = few_opaque(kGuCodes + li * 8 * kFewPairs);
    // the intermediate of the item before from the waves' partial sums
    int prev = -1;
    auto finish = [&](int par) MX_INLINE {
        const int g = prev / per, i0 = prev % per * width;
        const int i = threadIdx.x & (width - 1), t = threadIdx.x / width;
        const int slot = t < kFewT && prev >= 0 ? m.g.slot[g * kFewT + t] : -1;
        if (slot >= 0) {
            float gs = 0.f, us = 0.f;
#pragma unroll
            for (int w = 0; w < ks; ++w) {
                gs += red[par][(i >> 3) * ks + w][t][i & 7];
                us += red[par][(i >> 3) * ks + w][t][8 + (i & 7)];
            }
            p.a[(size_t)slot * p.I + i0 + i] = silu_mul(gs, us);
        }
    };
    auto body = [&](uint8_t (&st)[kFewWaves][kGuStage], auto par_c) MX_INLINE {
        constexpr int par = decltype(par_c)::value;
        wait_vmcnt<kGuLoads>();  // this item has landed; the next one may fly
        finish(par ^ 1);
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        u32x4 sc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            sc[i] = *reinterpret_cast<const u32x4*>(st[wave] + srow + 16 * i);
#pragma unroll
        for (int j = 0; j < kFewPairs; ++j) {
            const uint32_t own = j < cnt ? ~0u : 0u;  // zeros times 2^-127 in the steps past this wave's
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const u32x4 a = *reinterpret_cast<const u32x4*>(st[wave] + j * 2048 + few_at(li, 4 * u + lk));
                acc = mfma16_fp4(a, b[2 * j + u], acc, (sc[j >> 1][2 * (j & 1) + u] >> (8 * lk)) & own, sb[2 * j + u]);
            }
        }
        *reinterpret_cast<f32x4*>(&red[par][wave][li][4 * lk]) = acc;
        mx_barrier();
        issue(it + 2 * G, n, st);
        prev = it;
        it += G;
    };
    const int n_items = n * per;
    if (it < n_items) {
        int par;
        for (;;) {
            body(s0, std::integral_constant<int, 0>{});
            par = 0;
            if (it >= n_items) break;
            body(s1, std::integral_constant<int, 1>{});
            par = 1;
            if (it >= n_items) break;
        }
        finish(par);
    }
    wait_vmcnt<0>();
}

// ---------------------------------------------------------------- down + combine
constexpr int kDnCols = 32;                        // output columns of a workgroup, at most
constexpr int kDnUnit = kDnCols * 128 + kDnCols * 8;  // 256 of K for each: codes, then scales
constexpr int kDnLoads = kDnCols / 8 + 1;
constexpr int kSegK = 256 * kFewWaves;             // a segment of K: one unit per wave
constexpr int kActBytes = 41952;                   // 37 rows of a whole segment: a group (kFewT) fits

// kWhole: rows of act hold whole segments (I >= 2048); otherwise rows as narrow as I, so that more of them fit
template <bool kWhole>
__global__ __launch_bounds__(kFewThreads) void few_down_kernel(FewArgs p) {
    __shared__ __attribute__((aligned(1024))) uint8_t s0[kFewWaves][kDnUnit];
    __shared__ __attribute__((aligned(1024))) uint8_t s1[kFewWaves][kDnUnit];
    __shared__ __attribute__((aligned(1024))) uint8_t s2[kFewWaves][kDnUnit];
    __shared__ __attribute__((aligned(16))) uint8_t act[kActBytes];  // quantised rows of the intermediate
    __shared__ FewGroups m;
    __shared__ FewSum fs;
    static_assert(sizeof(float) * kFewWaves * kDnCols * (kFewT + 1) <= sizeof(act), "the last sums reuse act");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, lk = lane >> 4;
    const int rowb = p.I / 2, kb = p.I / kMxBlock, nk = p.I / 128, np = (nk + 1) / 2;
    const int nseg = kWhole ? (p.I + kSegK - 1) / kSegK : 1;
    // a row of act: a segment's codes, its scales, and a pad; reads of a half that is not there end in the slack
    const int segk = kWhole ? kSegK : p.I, pitch = segk / 2 + ((segk / kMxBlock + 31) & ~15);
    const int act_rows = (kActBytes - 128) / pitch, eights = segk / 8;
    const int h0 = blockIdx.x * p.cols, cols = min(p.cols, p.H - h0);
    const int S = p.T * p.k, sh = p.has_shared ? 1 : 0;
    {
        constexpr int kDwords = sizeof(FewGroups) / 4, kEach = (kDwords + kFewThreads - 1) / kFewThreads;
        uint32_t t[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            t[i] = reinterpret_cast<const uint32_t*>(p.groups)[min((int)threadIdx.x + i * kFewThreads, kDwords - 1)];
        const int s = min((int)threadIdx.x, S - 1);
        const int id = p.ids[s];
        const float w = p.topk_w[s];
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (threadIdx.x + i * kFewThreads < kDwords)
                reinterpret_cast<uint32_t*>(&m)[threadIdx.x + i * kFewThreads] = t[i];
        if (threadIdx.x < S) {
            fs.id[threadIdx.x] = id;
            fs.w[threadIdx.x] = w;
        }
    }
    mx_barrier();
    const int n = __builtin_amdgcn_readfirstlane(m.n);
    const int nsg = n * nseg;  // sub-groups: a segment of a group
    auto group_of = [&](int sg) MX_INLINE { return nseg == 1 ? sg : sg / nseg; };

    // A wave takes the K step ksi of its groups. Where I has fewer than eight, the waves left over take other groups:
    // by the expert's number, so that a token's sum does not depend on the other tokens' experts. (50 experts at H =
    // 2048, I = 128: 31 us with one wave at work, 14 with eight.)
    const int ks = kWhole || np > 4 ? 8 : np > 2 ? 4 : np, ksi = wave & (ks - 1), cls = wave / ks;
    uint64_t mine[3] = {};
    int counter = 0;
    if (!kWhole && ks < 8) {
#pragma unroll
        for (int b = 0; b < 3; ++b) {
            const int g = 64 * b + lane, e = g < n ? m.expert[g] : -2;
            mine[b] = __ballot(e != -2 && (e < 0 ? 0 : e & (kFewWaves / ks - 1)) == cls);
        }
    }
    auto next_sg = [&]() MX_INLINE {  // ascending; nsg and more: none left
        if (kWhole || ks == 8) return counter++;
        const int b = mine[0] ? 0 : mine[1] ? 1 : 2;
        const uint64_t set = mine[0] ? mine[0] : mine[1] ? mine[1] : mine[2];
        const int sg = set ? 64 * b + (int)__builtin_ctzll(set) : nsg;
        const uint64_t rest = set & (set - 1);
        mine[2] = b == 2 ? rest : mine[2];
        mine[1] = b == 1 ? rest : mine[1];
        mine[0] = b == 0 ? rest : mine[0];
        return __builtin_amdgcn_readfirstlane(sg);
    };

    // rows past cols are past the descriptors' end and read zeros
    const uint32_t wv = (uint32_t)((lane >> 3) * rowb + ksi * 128 + (((lane & 7) ^ (lane >> 3)) << 4));
    const uint32_t sv = (uint32_t)((lane >> 1) * kb + ksi * 8 + (lane & 1) * 4);
    auto expert_of = [&](int sg) MX_INLINE { return m.expert[group_of(min(sg, max(nsg - 1, 0)))]; };
    auto issue = [&](int sg, int expert, uint8_t (&st)[kFewWaves][kDnUnit]) MX_INLINE {
        const int g = group_of(sg), seg = sg - g * nseg;
        const bool on = sg < nsg && kFewWaves * seg + ksi < np;
        const bool shared = g < sh;
        const int e = shared || !on ? 0 : __builtin_amdgcn_readfirstlane(expert);
        const uint8_t* W = (shared ? p.ws2 : p.w2 + (size_t)e * p.H * rowb) + (size_t)h0 * rowb;
        const uint8_t* Ws = (shared ? p.ws2s : p.w2s + (size_t)e * p.H * kb) + (size_t)h0 * kb;
        const __amdgpu_buffer_rsrc_t wd = buffer_rsrc(W, on ? (uint32_t)cols * rowb : 0),
                                     sd = buffer_rsrc(Ws, on ? (uint32_t)cols * kb : 0);
        lds_buf4(sd, sv, (uint32_t)seg * (kSegK / kMxBlock), st[wave] + kDnCols * 128);
#pragma unroll
        for (int i = 0; i < kDnCols / 8; ++i)
            lds_buf16(wd, wv, (uint32_t)seg * (kSegK / 2) + (uint32_t)(8 * i * rowb), st[wave] + i * 1024);
        asm volatile("" ::: "memory");  // loads of different stages stay in order: the waits count them
    };
    // act holds the rows of the sub-groups [.., c_end): row_of(sg) - c_row on
    int c_end = 0, c_row = 0;
    auto row_of = [&](int sg) MX_INLINE {
        const int g = group_of(sg);
        return nseg * fs.pre[g] + (sg - g * nseg) * (sg < nsg ? __popc(m.mask[g]) : 0);
    };
    // The rows from sub-group sg on, as many whole sub-groups as fit, eight values per thread at a time. begin() loads
    // the first ones.
    int rows = 0;
    constexpr int kBatch = 4;
    f32x4 v[kBatch][2];
    int to[kBatch], scale_to[kBatch];  // where they go, -1: nowhere
    const __amdgpu_buffer_rsrc_t ad = buffer_rsrc(p.a, (uint32_t)((S + p.T) * p.I * 4));
    auto load_rows = [&](int i0) MX_INLINE {  // zeros past the last row and past I
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int i = i0 + q * kFewThreads, r = i / eights, e8 = i - r * eights;
            int pair = c_row + min(r, max(rows - 1, 0)), seg = 0;
            if (nseg > 1 && rows > 0) {  // without rows (no local pick, no shared expert) there are no pairs to look up
                const int g = fs.pair_group[pair / nseg], rem = pair - nseg * fs.pre[g], c = max(__popc(m.mask[g]), 1);
                seg = rem / c;
                pair = fs.pre[g] + rem - seg * c;
            }
            const int k0 = seg * kSegK + e8 * 8;
            const uint32_t off = r < rows && k0 < p.I ? (uint32_t)(fs.pair_slot[pair] * p.I + k0) * 4 : 0xffffff00u;
            v[q][0] = __builtin_bit_cast(f32x4, buffer_load16(ad, off, 0));
            v[q][1] = __builtin_bit_cast(f32x4, buffer_load16(ad, off, 16));
            to[q] = r < rows ? r * pitch + e8 * 4 : -1;
            scale_to[q] = r < rows && (e8 & 3) == 0 ? r * pitch + segk / 2 + (e8 >> 2) : -1;
        }
    };
    auto begin = [&](int sg) MX_INLINE {
        c_row = __builtin_amdgcn_readfirstlane(row_of(sg));
        const int to_sg = min(sg + 1 + lane, nsg);  // at most 64 of them
        const uint64_t fit = __ballot(sg + 1 + lane <= nsg && row_of(to_sg) - c_row <= act_rows);
        c_end = sg + __popcll(fit);
        rows = __builtin_amdgcn_readfirstlane(row_of(c_end)) - c_row;
        load_rows(threadIdx.x);
    };
    auto quantise = [&]() MX_INLINE {
        mx_barrier();  // the rows before have been read
#pragma unroll 1
        for (int i0 = threadIdx.x; i0 < rows * eights; i0 += kBatch * kFewThreads) {
            uint32_t code[kBatch], byte[kBatch];
            int at[kBatch], scale_at[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = v[q][i >> 2][i & 3];
                code[q] = mx_quantise8(f, byte[q]);
                at[q] = to[q];
                scale_at[q] = scale_to[q];
            }
            load_rows(i0 + kBatch * kFewThreads);
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                if (at[q] >= 0) *reinterpret_cast<uint32_t*>(act + at[q]) = code[q];
                if (scale_at[q] >= 0) act[scale_at[q]] = (uint8_t)byte[q];
            }
        }
        wait_vmcnt<0>();  // said once here, or the compiler says it in the loop, before its stages' reads
        mx_barrier();
    };

    int sg0 = next_sg(), sg1 = next_sg(), sg2 = next_sg();  // what the stages hold
    issue(sg0, expert_of(sg0), s0);
    issue(sg1, expert_of(sg1), s1);
    issue(sg2, expert_of(sg2), s2);
    sum_few_map(m, fs, n, p);
    begin(0);
    quantise();

    const uint32_t srow = few_opaque(kDnCols * 128 + li * 8);
    f32x4 total[2] = {};
    auto body = [&](int& sg, uint8_t (&st)[kFewWaves][kDnUnit]) MX_INLINE {
        while (sg >= c_end) {
            begin(c_end);
            quantise();
        }
        wait_vmcnt<2 * kDnLoads>();  // this unit has landed; the next two may fly
        const int g = group_of(sg), seg = sg - g * nseg;
        const int after = next_sg(), expert = expert_of(after);
        const int left = nk - 2 * (kFewWaves * seg + ksi);  // halves of this wave's unit that are there
        const uint32_t mask = m.mask[g];
        const bool on = left > 0 && mask >> li & 1;
        const int sg_row = row_of(sg) - c_row;
        const float w = fs.weight[g * kFewT + li];
        // a column that nobody picked multiplies row 0's values and is dropped
        const int row = on ? sg_row + __popc(mask & ((1u << li) - 1)) : 0;
        const uint8_t* ar = act + row * pitch + (left > 0 ? ksi * 128 : 0);
        const uint64_t as =
            *reinterpret_cast<const uint64_t*>(act + row * pitch + segk / 2 + (left > 0 ? ksi * 8 : 0)) >> (8 * lk);
        f32x4 acc[2] = {};
        uint64_t ws[2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
            ws[q] = *reinterpret_cast<const uint64_t*>(st[wave] + srow + 128 * q) >> (8 * lk);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            // past the end of K: scales of 2^-127 on both sides, and the codes are numbers whatever they are
            const uint32_t own = u < left ? 0xffu : 0u;
            const u32x4 b = *reinterpret_cast<const u32x4*>(ar + (4 * u + lk) * 16);
            const uint32_t sb = (uint32_t)(as >> (32 * u)) & own;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const u32x4 a = *reinterpret_cast<const u32x4*>(st[wave] + few_at(16 * q + li, 4 * u + lk));
                acc[q] = mfma16_fp4(a, b, acc[q], (uint32_t)(ws[q] >> (32 * u)) & own, sb);
            }
        }
        // a token that did not pick this expert takes nothing from it, not even a NaN
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int r = 0; r < 4; ++r) total[q][r] = on ? __builtin_fmaf(w, acc[q][r], total[q][r]) : total[q][r];
        asm volatile("" ::: "memory");
        wait_lds();  // this stage has been read
        asm volatile("" ::: "memory");
        issue(after, expert, st);
        sg = after;
    };
    for (;;) {
        if (sg0 >= nsg) break;
        body(sg0, s0);
        if (sg1 >= nsg) break;
        body(sg1, s1);
        if (sg2 >= nsg) break;
        body(sg2, s2);
    }
    while (c_end < nsg) {  // the other waves' rows: all of them meet at the barriers
        begin(c_end);
        quantise();
    }
    wait_vmcnt<0>();
    mx_barrier();  // act is free
    float(*red)[kDnCols][kFewT + 1] = reinterpret_cast<float(*)[kDnCols][kFewT + 1]>(act);
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][16 * q + 4 * lk + r][li] = total[q][r];
    __syncthreads();
    const int c = threadIdx.x & 31, t = threadIdx.x >> 5;
    if (t < p.T && c < cols) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) s += red[w][c][t];
        p.out[(size_t)t * p.H + h0 + c] = (uint16_t)f32_to_bf16_bits(s);
    }
}

struct FewWs {
    FewGroups* groups;
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
    r.groups = (FewGroups*)take(sizeof(FewGroups));
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
        const moe_status r = launch_route_logits_rows(x, w_router, bias, T, w->H, E, s.logits, st);
        if (r) return r;
    }
    FewArgs p{};
    p.x = (const uint16_t*)x;
    p.logits = w_router ? s.logits : nullptr;
    p.ids = topk_ids;
    p.topk_w = topk_w;
    p.T = T;
    p.k = k;
    p.E = E;
    p.scoring = scoring;
    p.renorm = renorm;
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
    p.groups = s.groups;
    p.a = s.a;
    p.out = (uint16_t*)out;
    const int cu = device_info().cu_count;
    // 8 columns are one load: as many workgroups as the CUs, or 32 columns each
    p.cols = std::min(kDnCols, (int)align_up((size_t)(w->H + cu - 1) / cu, 8));
    // As few waves to an item's K as their stages allow, and so as many columns (at most 32: a thread for each and each
    // token): an item's sums and barrier cost 1.5 us whatever it loads. 50 experts at H = 512, I = 2048 take 78 us with
    // 8 columns an item and 26 with 32, 38 experts at H = 1024 64 and 25.
    const int ks = w->H <= 2 * 256 * kFewPairs ? 2 : w->H <= 4 * 256 * kFewPairs ? 4 : 8;
    const long items = ((long)std::min(T * k, w->E_local) + p.has_shared) * (w->I / (8 * kFewWaves / ks));
    auto gate_up = ks == 2 ? few_gate_up_kernel<2> : ks == 4 ? few_gate_up_kernel<4> : few_gate_up_kernel<8>;
    hipLaunchKernelGGL(gate_up, dim3((int)std::min<long>(cu, items)), dim3(kFewThreads), 0, st, p);
    const moe_status r = check_launch("few_gate_up_kernel");
    if (r) return r;
    auto down = w->I >= kSegK ? few_down_kernel<true> : few_down_kernel<false>;
    hipLaunchKernelGGL(down, dim3((w->H + p.cols - 1) / p.cols), dim3(kFewThreads), 0, st, p);
    return check_launch("few_down_kernel");
}

}  // namespace moe
