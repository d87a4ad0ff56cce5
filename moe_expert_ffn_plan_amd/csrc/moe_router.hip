// Router product: logits[t, e] = sum_k x[t, k] w[e, k] on BF16 MFMA with FP32 accumulators.
//
// Products of two BF16 values are exact in FP32.  An FP32 weight is split once, ahead of all calls, into
// three BF16 parts by truncation (8 of its 24 significant bits each, so the parts add up to it exactly);
// the product then runs three times as many matrix instructions, still 5 times the rate of FP32 ones.
//
// Weights are laid out once in the order of the matrix instruction's operand: one 1 KiB block per 16
// experts, 32 columns and part; lane l of it holds expert l % 16, columns 8 (l / 16) .. + 8.
// V_MFMA_F32_16X16X32_BF16 with A = weights, B = x: lane l of the result holds token l % 16 and the four
// experts 4 (l / 16) .. + 4, neighbours in a logits row.
#include "moe_internal.h"

#include <type_traits>

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

// One thread per 16 bytes of one part: 8 columns of one expert.
template <int TYPE>
__global__ __launch_bounds__(kThreads) void router_prepare_kernel(const void* __restrict__ w, int H, int E,
                                                                  int64_t slots, uint8_t* __restrict__ out) {
    const int64_t s = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (s >= slots) return;
    const int lane = (int)(s & 63), KT = H / 32;
    const int64_t blk = s >> 6;
    const int e = (int)(blk / KT) * 16 + (lane & 15);
    const int k = (int)(blk % KT) * 32 + (lane >> 4) * 8;
    constexpr int P = TYPE == MOE_F32 ? 3 : 1;
    uint16_t part[P][8] = {};
    if (e < E) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t i = (int64_t)e * H + k + j;
            if constexpr (TYPE == MOE_F32) {
                float v = static_cast<const float*>(w)[i];
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const uint32_t top = __float_as_uint(v) & 0xFFFF0000u;
                    part[p][j] = (uint16_t)(top >> 16);
                    v -= __uint_as_float(top);
                }
            } else {
                part[0][j] = static_cast<const uint16_t*>(w)[i];
            }
        }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
        uint4 o;
        uint32_t* q = &o.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = (uint32_t)part[p][2 * j] | ((uint32_t)part[p][2 * j + 1] << 16);
        reinterpret_cast<uint4*>(out)[(blk * P + p) * 64 + lane] = o;
    }
}

// Stores four neighbouring logits of token t, experts e .. e + 4.
__device__ __forceinline__ void store_logits(float* logits, int E, int64_t t, int e, v4f v) {
    float* p = logits + t * E + e;
    if (E % 4 == 0) {
        if (e < E) *reinterpret_cast<v4f*>(p) = v;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (e + j < E) p[j] = v[j];
    }
}

// ---- LDS DMA and waits (the compiler does not count what inline assembly issues; each kernel waits itself)

// Lane l reads 16 bytes at its own address and writes them at LDS address lds + 16 l.  With the non-temporal hint,
// which keeps the weights in the L2, for an x that the memory-side cache (256 MB, which the hint passes by) does
// not hold next to the rest of a layer: 8192 x 7168 x 256 44.2 us, 47.1 without; 16384: 71.5, 76.3.
constexpr int64_t kStreamBytes = 1 << 26;
__device__ __forceinline__ void dma16_stream(uint64_t addr, uint32_t lds) {
    asm volatile("global_load_lds_dwordx4 %0, off nt" ::"v"(addr), "{m0}"(lds) : "memory");
}
// Without it for a smaller x, that the norm wrote just before: 4096 x 7168 x 256 23.9 us, 30.6 with it; 2048 16.4,
// 20.9; the small kernel at 16 tokens 5.5, 11.0.
__device__ __forceinline__ void dma16(uint64_t addr, uint32_t lds) {
    asm volatile("global_load_lds_dwordx4 %0, off" ::"v"(addr), "{m0}"(lds) : "memory");
}
// The same at a wave-uniform base and a 32-bit offset per lane, kept in the L2.
__device__ __forceinline__ void dma16_at(uint32_t off, const void* base, uint32_t lds) {
    asm volatile("global_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_and_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)p);
}

// The x operand lies in LDS as rows of CH 16-byte chunks (64 or 128 columns), chunk c of row r at a place
// that gives the 16 rows that a ds_read_b128 takes at one chunk 16 different slots modulo the 256 bytes of the
// banks: rows of 256 bytes swap chunks by r, rows of 128 bytes, of which two fit, by r >> 1.  (Rows of 256
// bytes by r >> 1 were two-way conflicts, half of the LDS time.)  Reading x into registers directly puts
// neighbouring lanes on different rows, which the address unit takes one lane at a time (a kernel of 16-token
// tiles at 128 x 7168 x 256: 10.0 us against 7.1 through LDS).
template <int CH>
__device__ __forceinline__ int swizzle(int row, int chunk) {
    static_assert(CH == 8 || CH == 16, "128 or 256 bytes");
    return CH == 16 ? chunk ^ (row & 15) : chunk ^ ((row >> 1) & 7);
}

// The sum over the parts of an FP32 weight: the first parts' products in one accumulator, those of the
// other two in another, so that the small terms do not round the large sum twice more per step.
template <int P, int N, int M>
struct Sums {
    static constexpr int SETS = P > 1 ? 2 : 1;
    v4f v[SETS][N][M];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int s = 0; s < SETS; ++s)
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int m = 0; m < M; ++m) v[s][n][m] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    __device__ __forceinline__ void add(int p, int n, int m, bf16x8 w, bf16x8 x) {
        v4f& c = v[p > 0 ? SETS - 1 : 0][n][m];
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, c, 0, 0, 0);
    }
    __device__ __forceinline__ v4f total(int n, int m) const {
        return SETS == 1 ? v[0][n][m] : v[0][n][m] + v[SETS - 1][n][m];
    }
};

// ---- few tokens or columns: one workgroup per 16 tokens and 16 experts, in one launch
//
// The 16 waves split the columns, wave w taking every 16th run of 64, with kRuns runs in flight (x through its own
// piece of LDS, the weights straight into registers, 1 KiB a load), and add up through LDS in the order of the
// waves.  Bound by latency, and by the L1 where rows are long: a workgroup takes 32 H (1 + parts) bytes through it
// (16 x 7168 x 256: 5.5 us; 128 rows: 7.1; 128 x 2048 x 512: 4.1).  Each run's successor issued as soon as its place is
// free, instead of kRuns at a time, gained nothing (7.1 to 7.8 at 128 rows).
constexpr int kSmallTokens = 16, kSmallWaves = 16, kRuns = 4;

template <int P>
__global__ __launch_bounds__(kSmallWaves * 64) void router_small_kernel(RouterArgs a) {
    constexpr int RUN = kSmallTokens * 128;  // bytes of one run of x
    __shared__ __align__(1024) uint8_t lds[kSmallWaves * kRuns * RUN];
    static_assert(kRuns * RUN >= 1024, "holds the waves' sums");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int KT = a.H / 32, runs = (KT + 1) / 2;
    const int r16 = lane & 15, q = lane >> 4, m0 = blockIdx.y * kSmallTokens;
    uint64_t xp[2];                          // transfer i: rows 8 i .. 8 i + 8 of the run
    int xc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = i * 8 + (lane >> 3);
        xc[i] = swizzle<8>(row, lane & 7);
        xp[i] = reinterpret_cast<uint64_t>(a.x + (int64_t)min(m0 + row, a.T - 1) * a.x_stride + xc[i] * 8);
    }
    const uint8_t* wp = a.w + (int64_t)blockIdx.x * KT * P * 1024;
    Sums<P, 1, 1> acc;
    acc.clear();
    const uint32_t mine = lds_addr(lds) + wave * kRuns * RUN;
    const uint8_t* xs = lds + wave * kRuns * RUN;
    for (int r0 = wave; r0 < runs; r0 += kRuns * kSmallWaves) {
        bf16x8 w[kRuns][2][P];
#pragma unroll
        for (int u = 0; u < kRuns; ++u) {
            const int r = r0 + u * kSmallWaves;
            if (r >= runs) break;
            // a last run of 32 columns: the missing chunks read the run's first, and are not multiplied
            const bool half = 2 * r + 1 >= KT;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                dma16(xp[i] + (int64_t)r * 128 - (half && xc[i] >= 4 ? xc[i] * 16 : 0),
                             mine + u * RUN + i * 1024);
        }
#pragma unroll
        for (int u = 0; u < kRuns; ++u) {
            const int r = r0 + u * kSmallWaves;
            if (r >= runs) break;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int p = 0; p < P; ++p)
                    w[u][j][p] = *reinterpret_cast<const bf16x8*>(
                        wp + ((int64_t)min(2 * r + j, KT - 1) * P + p) * 1024 + lane * 16);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int u = 0; u < kRuns; ++u) {
            const int r = r0 + u * kSmallWaves;
            if (r >= runs) break;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (2 * r + j >= KT) break;
                const bf16x8 x = *reinterpret_cast<const bf16x8*>(xs + u * RUN + r16 * 128 + swizzle<8>(r16, j * 4 + q) * 16);
#pragma unroll
                for (int p = 0; p < P; ++p) acc.add(p, 0, 0, w[u][j][p], x);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // x is read before the next runs overwrite it
    }
    __syncthreads();
    v4f(*part)[64] = reinterpret_cast<v4f(*)[64]>(lds);
    part[wave][lane] = acc.total(0, 0);
    __syncthreads();
    if (wave == 0) {
        v4f sum = part[0][lane];
#pragma unroll
        for (int w = 1; w < kSmallWaves; ++w) sum += part[w][lane];
        if (m0 + r16 < a.T) store_logits(a.logits, a.E, m0 + r16, blockIdx.x * 16 + q * 4, sum);
    }
}

// ---- many tokens: tiles of BM tokens x 64 NF experts over a range of K-steps of BK columns
//
// Four producer waves stream x into an LDS ring of NS stages and do nothing else; four consumer waves, one
// per SIMD, each own 16 NF experts and all BM tokens.  A consumer reads its weights from the L2 straight
// into registers (they lie in operand order, so LDS would only add a round trip), one K-step ahead, and x
// from the ring, four fragments ahead of the matrix instructions.  One barrier per step publishes a stage
// and frees the one before it; producers wait for their own transfers ahead of it, consumers for their LDS
// reads, and a consumer has the next step's first fragments in flight before it starts the last products
// of its step.
// Where it goes (16384 x 7168 x 256, 128 x 256 tiles in two splits, 62 us of the call's 70): the matrix cores
// are busy for 48% of the CUs' 121,000 clocks; x alone streams in 35 us and the products alone, with both
// operands in the L2, take 45.  The L1 takes loads in order at about 50 bytes a clock, so the weights wait
// behind x from memory: a CU moves 24 KiB per 32 columns, 480 of the 512 clocks of its matrix instructions.
// 64 x 256 tiles need no second split but move 20 KiB for half of the products and take 75 us.  Writing the
// result (all workgroups end together) and adding the splits take the other 20 us.
template <int BM_, int NF_, int NS_, int BK_, int P_>
struct Tile {
    static constexpr int BM = BM_, NF = NF_, NS = NS_, BK = BK_, P = P_;
    static constexpr int CW = 4, PW = 4, THREADS = (CW + PW) * 64, BN = NF * CW * 16;
    static constexpr int KS = BK / 32, MT = BM / 16, CH = BK / 8;       // 16-byte chunks per row and step
    static constexpr int STAGE = BM * BK * 2, PER = STAGE / 1024 / PW;  // transfers per producer and stage
    static constexpr int GS = MT < 4 ? MT : 4, GPK = MT / GS, NG = KS * GPK;  // fragment groups of a step
    static_assert((BK == 64 || BK == 128) && MT % GS == 0 && NG % 2 == 0, "whole runs; two fragment buffers alternate");
    static_assert(STAGE % (1024 * PW) == 0 && NS >= 2 && NS * STAGE <= 160 * 1024, "the ring");
    static_assert(PER * (NS - 2) < 63, "vmcnt counts to 63");
};

struct TileArgs {
    RouterArgs r;
    int m_tiles, n_tiles, splits, steps;  // K-steps in all
    bool stream_x;
};

template <class C>
__global__ __launch_bounds__(C::THREADS) void router_tile_kernel(TileArgs a) {
    __shared__ __align__(1024) uint8_t ring[C::NS * C::STAGE];
    // XCD b % 8 takes a contiguous run of the list [split][m tile][n tile]: what shares x or a part of the
    // weights runs side by side on one L2
    const int total = a.m_tiles * a.n_tiles * a.splits, share = (total + 7) / 8;
    const int v = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
    if (v >= total) return;  // the grid is 8 * share workgroups
    const int split = v / (a.m_tiles * a.n_tiles), mn = v % (a.m_tiles * a.n_tiles);
    const int m0 = mn / a.n_tiles * C::BM, n0 = mn % a.n_tiles * C::BN;
    const int s_begin = (int)((int64_t)a.steps * split / a.splits);
    const int s_end = (int)((int64_t)a.steps * (split + 1) / a.splits);
    const int n_steps = s_end - s_begin;  // >= 1: splits <= steps
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int KT = a.r.H / 32;

    if (wave >= C::CW) {
        const int pw = wave - C::CW;
        const uint32_t ring0 = lds_addr(ring);
        uint64_t src[C::PER];
        int chunk[C::PER];
#pragma unroll
        for (int i = 0; i < C::PER; ++i) {
            const int slot = (pw + i * C::PW) * 64 + lane, row = slot / C::CH;
            chunk[i] = swizzle<C::CH>(row, slot % C::CH);
            src[i] = reinterpret_cast<uint64_t>(a.r.x + (int64_t)min(m0 + row, a.r.T - 1) * a.r.x_stride + chunk[i] * 8);
        }
        auto issue = [&](int step, int stage) {
            // a last step of fewer columns: the missing chunks read the step's first, and are not multiplied
            const int valid = (KT - step * C::KS) * 4;
            auto all = [&](auto dma) {
#pragma unroll
                for (int i = 0; i < C::PER; ++i)
                    dma(src[i] + (int64_t)step * (C::BK * 2) - (chunk[i] >= valid ? chunk[i] * 16 : 0),
                        ring0 + stage * C::STAGE + (pw + i * C::PW) * 1024);
            };
            if (a.stream_x) all(dma16_stream);  // (asked at each transfer: 1.5% at 16384 x 7168 x 256)
            else all(dma16);
        };
#pragma unroll
        for (int s = 0; s < C::NS - 1; ++s)
            if (s < n_steps) issue(s_begin + s, s);
        int stage = 0;
        for (int s = 0; s < n_steps; ++s) {
            if (n_steps - 1 - s >= C::NS - 2) wait_and_barrier<(C::NS - 2) * C::PER>();
            else wait_and_barrier<0>();
            if (s + C::NS - 1 < n_steps) issue(s_begin + s + C::NS - 1, stage == 0 ? C::NS - 1 : stage - 1);
            stage = stage == C::NS - 1 ? 0 : stage + 1;
        }
        return;
    }

    const uint8_t* wp[C::NF];  // wave-uniform; blocks past the last read the last, and are not stored
#pragma unroll
    for (int n = 0; n < C::NF; ++n)
        wp[n] = a.r.w + (int64_t)min(n0 / 16 + wave * C::NF + n, (a.r.E + 15) / 16 - 1) * KT * C::P * 1024;
    const uint32_t lane16 = lane * 16;
    bf16x8 w[C::KS][C::P][C::NF];
    auto load = [&](int k, int p, int n) {
        return *reinterpret_cast<const bf16x8*>(wp[n] + ((int64_t)min(k, KT - 1) * C::P + p) * 1024 + lane16);
    };
    bf16x8 xg[2][C::GS];
    const int r16 = lane & 15, q = lane >> 4;
    uint32_t x_at[C::KS];
#pragma unroll
    for (int ks = 0; ks < C::KS; ++ks) x_at[ks] = r16 * (C::BK * 2) + swizzle<C::CH>(r16, ks * 4 + q) * 16;
    auto read = [&](const uint8_t* stage, int g, int i) {  // fragment i of group g
        return *reinterpret_cast<const bf16x8*>(stage + x_at[g / C::GPK] + (g % C::GPK * C::GS + i) * 16 * (C::BK * 2));
    };
    Sums<C::P, C::NF, C::MT> acc;
    acc.clear();
    auto multiply = [&](int g, int p, int n) {
#pragma unroll
        for (int i = 0; i < C::GS; ++i)
            acc.add(p, n, g % C::GPK * C::GS + i, w[g / C::GPK][p][n], xg[g & 1][i]);
    };

#pragma unroll
    for (int k = 0; k < C::KS; ++k)
#pragma unroll
        for (int p = 0; p < C::P; ++p)
#pragma unroll
            for (int n = 0; n < C::NF; ++n) w[k][p][n] = load(s_begin * C::KS + k, p, n);
    asm volatile("s_barrier" ::: "memory");
#pragma unroll
    for (int i = 0; i < C::GS; ++i) xg[0][i] = read(ring, 0, i);
    int stage = 0;
    for (int s = 0; s < n_steps - 1; ++s) {
        const int next = stage == C::NS - 1 ? 0 : stage + 1;
#pragma unroll
        for (int g = 0; g < C::NG; ++g) {
            const uint8_t* from = ring + (g < C::NG - 1 ? stage : next) * C::STAGE;
            if (g == C::NG - 1) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            // a load takes its wave's issue slot for as long as the L1 needs to take its kilobyte: one after
            // the last products of each register that it fills, and the LDS reads between products as well
#pragma unroll
            for (int u = 0; u < C::P * C::NF; ++u) {
                const int p = u / C::NF, n = u % C::NF;
#pragma unroll
                for (int i = u * C::GS / (C::P * C::NF); i < (u + 1) * C::GS / (C::P * C::NF); ++i)
                    xg[(g + 1) & 1][i] = read(from, g < C::NG - 1 ? g + 1 : 0, i);
                __builtin_amdgcn_sched_barrier(0);
                multiply(g, p, n);
                if (g % C::GPK == C::GPK - 1)
                    w[g / C::GPK][p][n] = load((s_begin + s + 1) * C::KS + g / C::GPK, p, n);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        stage = next;
    }
    const int valid = min(C::KS, KT - (s_end - 1) * C::KS);
#pragma unroll
    for (int g = 0; g < C::NG; ++g) {
        if (g / C::GPK >= valid) break;
        if (g < C::NG - 1) {
#pragma unroll
            for (int i = 0; i < C::GS; ++i) xg[(g + 1) & 1][i] = read(ring + stage * C::STAGE, g + 1, i);
        }
#pragma unroll
        for (int u = 0; u < C::P * C::NF; ++u) multiply(g, u / C::NF, u % C::NF);
    }
    float* out = a.splits > 1 ? a.r.partial + (int64_t)split * a.r.T * a.r.E : a.r.logits;
#pragma unroll
    for (int m = 0; m < C::MT; ++m) {
        const int t = m0 + m * 16 + r16;
        if (t >= a.r.T) continue;
#pragma unroll
        for (int n = 0; n < C::NF; ++n)
            store_logits(out, a.r.E, t, n0 + (wave * C::NF + n) * 16 + q * 4, acc.total(n, m));
    }
}

// ---- very many tokens at 257 to 384 experts: tiles of 256 tokens x 384 experts
//
// Held back by the clock (65536 x 7168 x 384 runs the tile kernel's matrix instructions at 1.7 GHz), so the
// tile that moves the fewest bytes per product wins: 288 us against 343 for 128 x 192 (tiles of 256 x 256 at
// 256 experts do not: 244 against 234).  Eight waves, two per SIMD, each own 128 tokens x 96 experts in 192
// registers; both operands come through a ring of four 32-column stages in all of the LDS, transferred by
// the waves themselves.  A wave reads its six weight fragments once per stage and its eight of x one by one,
// two ahead; the barrier that publishes the next stage stands ahead of the last fragment's products, among
// which the next weights replace the old.  Halves of x's 128-byte lines arrive a step apart, so x is kept in
// the L2 (with the non-temporal hint 1.6 times its bytes came from memory: 312 us).
struct Big {
    static constexpr int BM = 256, NF = 6, WN = 4, BN = 16 * NF * WN, BK = 32, WAVES = 8, MT = 8, NS = 4;
    static constexpr int X_BYTES = BM * 64, STAGE = X_BYTES + BN * 64;
    static constexpr int PER = STAGE / 1024 / WAVES, X_PER = X_BYTES / 1024 / WAVES, W_PER = PER - X_PER;
    static_assert(NS * STAGE <= 160 * 1024 && PER * 1024 * WAVES == STAGE && PER < MT, "the ring");
};
constexpr int64_t kBigMaxStride = 1 << 22;  // a tile's rows within 32-bit byte offsets

// Chunk c of 64-byte row r lies at c ^ quarter(r): no bank conflicts counted (with (r >> 2) & 3 for quarter(r)
// half of the reads of x conflicted).
__device__ __forceinline__ int quarter(int row) { return (0x78 >> (((row >> 2) & 3) * 2)) & 3; }

__global__ __launch_bounds__(Big::WAVES * 64) void router_big_kernel(RouterArgs a) {
    using C = Big;
    __shared__ __align__(1024) uint8_t ring[C::NS * C::STAGE];
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int steps = a.H / C::BK, m0 = blockIdx.x * C::BM;

    uint32_t x_off[C::X_PER];  // transfers of 16 rows
#pragma unroll
    for (int i = 0; i < C::X_PER; ++i) {
        const int row = (wave + i * C::WAVES) * 16 + (lane >> 2);
        const int c = (lane & 3) ^ quarter(row);
        x_off[i] = (uint32_t)((min(m0 + row, a.T - 1) - m0) * (int)a.x_stride + c * 8) * 2u;
    }
    const uint8_t* x0 = reinterpret_cast<const uint8_t*>(a.x + (int64_t)m0 * a.x_stride);
    const uint8_t* w0[C::W_PER];  // blocks past the last read the last, and are not stored
#pragma unroll
    for (int i = 0; i < C::W_PER; ++i)
        w0[i] = a.w + (int64_t)min(wave + i * C::WAVES, (a.E + 15) / 16 - 1) * steps * 1024;
    const uint32_t lane16 = lane * 16;
    const uint32_t ring0 = lds_addr(ring);
    auto issue = [&](int i, int step, int stage) {
        const uint32_t to = ring0 + stage * C::STAGE + (wave + i * C::WAVES) * 1024;
        if (i < C::X_PER) dma16_at(x_off[i], x0 + (int64_t)step * 64, to);
        else dma16_at(lane16, w0[i < C::X_PER ? 0 : i - C::X_PER] + (int64_t)step * 1024, to);
    };
    const uint32_t x_at = (wm * 128 + r16) * 64 + (q ^ quarter(r16)) * 16;
    auto read_x = [&](int stage, int m) {
        return *reinterpret_cast<const bf16x8*>(ring + stage * C::STAGE + x_at + m * 1024);
    };
    auto read_w = [&](int stage, int n) {
        return *reinterpret_cast<const bf16x8*>(ring + stage * C::STAGE + C::X_BYTES + (wn * C::NF + n) * 1024 + lane16);
    };
    Sums<1, C::NF, C::MT> acc;
    acc.clear();
#pragma unroll
    for (int s = 0; s < C::NS - 1; ++s)
        if (s < steps) {
#pragma unroll
            for (int i = 0; i < C::PER; ++i) issue(i, s, s);
        }
    if (steps >= C::NS - 1) wait_and_barrier<(C::NS - 2) * C::PER>();
    else wait_and_barrier<0>();
    bf16x8 w[C::NF], x[3];
#pragma unroll
    for (int n = 0; n < C::NF; ++n) w[n] = read_w(0, n);
    x[0] = read_x(0, 0);
    x[1] = read_x(0, 1);
    int stage = 0, freed = C::NS - 1;
    // more: a stage is left to be transferred; last: none to be read
    auto step = [&](int s, auto more, auto last) {
        constexpr bool MORE = decltype(more)::value, LAST = decltype(last)::value;
        const int next = stage == C::NS - 1 ? 0 : stage + 1;
#pragma unroll
        for (int m = 0; m < C::MT; ++m) {
            if (m + 2 < C::MT) x[(m + 2) % 3] = read_x(stage, m + 2);
            if constexpr (MORE)
                if (m < C::PER) issue(m, s + C::NS - 1, freed);
            __builtin_amdgcn_sched_barrier(0);
            if (m < C::MT - 1 || LAST) {
#pragma unroll
                for (int n = 0; n < C::NF; ++n) acc.add(0, n, m, w[n], x[m % 3]);
            } else {
                if constexpr (MORE) wait_and_barrier<(C::NS - 2) * C::PER>();
                else wait_and_barrier<0>();
                static_assert((C::MT - 1) % 3 == 1, "x[0] and x[2] are free here");
                x[0] = read_x(next, 0);
#pragma unroll
                for (int n = 0; n < C::NF; ++n) {
                    acc.add(0, n, m, w[n], x[m % 3]);
                    w[n] = read_w(next, n);
                    __builtin_amdgcn_sched_barrier(0);
                }
                x[1] = read_x(next, 1);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        stage = next;
        freed = freed == C::NS - 1 ? 0 : freed + 1;
    };
    int s = 0;
    for (; s + C::NS - 1 < steps; ++s) step(s, std::true_type{}, std::false_type{});
    for (; s < steps - 1; ++s) step(s, std::false_type{}, std::false_type{});
    step(s, std::false_type{}, std::true_type{});
#pragma unroll
    for (int m = 0; m < C::MT; ++m) {
        const int t = m0 + wm * 128 + m * 16 + r16;
        if (t >= a.T) continue;
#pragma unroll
        for (int n = 0; n < C::NF; ++n) store_logits(a.logits, a.E, t, (wn * C::NF + n) * 16 + q * 4, acc.total(n, m));
    }
}

// Sums the splits' partial products [splits][n], in their order; 8 loads in flight per thread, of V floats
// (4 where n is a multiple of 4 and large; 1 keeps a small sum on many CUs).
template <int V>
__global__ __launch_bounds__(kThreads) void router_reduce_kernel(const float* __restrict__ part, int splits, int64_t n,
                                                                 float* __restrict__ out) {
    typedef float vec __attribute__((ext_vector_type(V)));
    const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * V;
    if (i >= n) return;
    vec sum = {};
    for (int s0 = 0; s0 < splits; s0 += 8) {
        vec v[8];
#pragma unroll
        for (int s = 0; s < 8; ++s)
            if (s0 + s < splits) v[s] = *reinterpret_cast<const vec*>(part + (s0 + s) * n + i);
#pragma unroll
        for (int s = 0; s < 8; ++s)
            if (s0 + s < splits) sum += v[s];
    }
    *reinterpret_cast<vec*>(out + i) = sum;
}

// ---- which kernel
//
// The one with the least estimated time (microseconds of the whole call), out of all tiles and of 1, 2, 4, 8 and
// as many splits as fill the CUs:
//   2.4 + rounds (0.84 + (H / 32 / splits) cost (1 + 0.44 share of the CUs in use))
//       + (2.2 + 0.46 per MB of partial sums where there are splits), at least 4.1, or 6.6 with the second launch.
// cost is a tile's time per 32 columns on an idle chip.  The constants are a fit to 3800 timings (T 8 .. 40000,
// H 1024 .. 7168, E 32 .. 1024, every tile and several splits; operands that do not lie in the L2); over their 473
// shapes its choice takes 1.3% more than the fastest on average, where borders on the number of tiles alone took
// 15% more.  Both sides of some borders:
//   128 x 2048 x 512: one launch of 16 x 16 tiles 4.1, 32 x 64 in 4 splits 6.9; 64 x 7168 x 256: 6.5, 7.0; 256 x 7168
//   x 256: 8.6, 7.9.  2048 x 1024 x 256: 32 x 64 whole 5.3, 64 x 128 in two splits 10.2.
//   512 x 7168 x 256: 32 x 64 in 4 splits 10.2, 32 x 128 in 8 9.7; 2048: 64 x 64 in two 18.2, 64 x 128 in four 16.3;
//   8192: 64 x 128 46, 128 x 256 in four 44; 16384: 91, 71 in two.
//   40000 x 7168 x 384: 128 x 192 249, 256 x 384 218; 8192: 49, 64.
//   FP32 weights, H 7168, E 256: T 512 32 x 64 in 4 splits 12.8, 64 x 64 in 8 14.1; T 1024: 21.1 in 2, 16.4 in 4;
//   T 16384: 64 x 128 178, 128 x 128 134.
constexpr int kCus = 256;
constexpr int kSmallMost = 1024;  // tokens, as measured; a grid axis holds 16 times 65535

enum Kernel { kSmall, kTile32x64, kTile32x128, kTile64x64, kTile64x128, kTile128x128, kTile128x192, kTile128x256, kBig };
struct Tiling {
    Kernel kernel;
    int bm, bn, bk;
    double cost;  // us
};
constexpr Tiling kBf16[] = {
    {kSmall, 16, 16, 64, 0.014},       {kTile32x64, 32, 64, 128, 0.052},    {kTile64x64, 64, 64, 128, 0.095},
    {kTile32x128, 32, 128, 128, 0.075}, {kTile64x128, 64, 128, 128, 0.120},  {kTile128x192, 128, 192, 128, 0.250},
    {kTile128x256, 128, 256, 128, 0.300}, {kBig, Big::BM, Big::BN, Big::BK, 0.865}};
constexpr Tiling kF32[] = {
    {kSmall, 16, 16, 64, 0.028}, {kTile32x64, 32, 64, 128, 0.095}, {kTile64x64, 64, 64, 128, 0.140},
    {kTile64x128, 64, 128, 64, 0.235}, {kTile128x128, 128, 128, 64, 0.385}};

// Tokens of a launch: tiles of 64 x 128 or more, and of 64 x 64 up to 64 experts, then fit one for any number of experts,
// and none of them is split (more tiles than CUs).
constexpr int kLaunchRows = 1 << 24;

int div_up(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <int P>
hipError_t launch_small(const RouterArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)div_up(a.E, 16), (unsigned)div_up(a.T, kSmallTokens));
    hipLaunchKernelGGL(router_small_kernel<P>, grid, dim3(kSmallWaves * 64), 0, stream, a);
    return hipGetLastError();
}

template <class C>
hipError_t launch_tile(const RouterArgs& r, int splits, hipStream_t stream) {
    const TileArgs a{r, div_up(r.T, C::BM), div_up(r.E, C::BN), splits, div_up(r.H, C::BK),
                     (int64_t)r.T * r.H * 2 > kStreamBytes};
    const int64_t total = (int64_t)a.m_tiles * a.n_tiles * splits;
    hipLaunchKernelGGL(router_tile_kernel<C>, dim3((unsigned)div_up(total, 8) * 8), dim3(C::THREADS), 0, stream, a);
    if (splits > 1) {
        const int64_t n = (int64_t)r.T * r.E;
        if (n % 4 == 0 && n >= (int64_t)4 * kThreads * kCus)
            hipLaunchKernelGGL(router_reduce_kernel<4>, dim3((unsigned)div_up(n, 4 * kThreads)), dim3(kThreads), 0, stream,
                               r.partial, splits, n, r.logits);
        else
            hipLaunchKernelGGL(router_reduce_kernel<1>, dim3((unsigned)div_up(n, kThreads)), dim3(kThreads), 0, stream,
                               r.partial, splits, n, r.logits);
    }
    return hipGetLastError();
}

bool allowed(const Tiling& c, int E) {
    if (c.kernel == kBig) return E > 256 && E <= Big::BN;
    return c.bn <= 64 || c.bn < 2 * E;  // the others are not measured
}

// f(s) for each number of splits to choose from: two K-steps at least, two workgroups a CU at most.
template <class F>
void each_split(const Tiling& c, int64_t tiles, int H, F&& f) {
    f(1);
    if (c.kernel == kSmall || c.kernel == kBig || tiles > kCus) return;
    const int steps = div_up(H, c.bk);
    const int fill = std::min(kCus / (int)tiles, steps / 4);  // four K-steps at least
    for (const int s : {2, 4, 8, fill})
        if (s > 1 && 2 * s <= steps && s * tiles <= 2 * kCus) f(s);
}
constexpr int64_t kMostPartial = 1 << 26;  // floats of partial sums

template <class F>
void each_tiling(int parts, F&& f) {
    if (parts == 3)
        for (const Tiling& c : kF32) f(c);
    else
        for (const Tiling& c : kBf16) f(c);
}

}  // namespace

RouterChoice choose_router(int T, int H, int E, int parts) {
    RouterChoice best{kSmall, kSmallTokens, 16, 1};
    if (T == 0) return best;
    T = std::min(T, kLaunchRows);
    double least = INFINITY;
    each_tiling(parts, [&](const Tiling& c) {
        if (!allowed(c, E) || (c.kernel == kSmall && T > kSmallMost)) return;
        const int64_t tiles = (int64_t)div_up(T, c.bm) * div_up(E, c.bn);
        if (tiles > 1 << 22) return;  // times 512 threads: what a launch takes
        each_split(c, tiles, H, [&](int s) {
            if (s > 1 && (int64_t)s * T * E > kMostPartial) return;
            const int groups = (int)tiles * s;
            const double used = (double)std::min(groups, kCus) / kCus;
            double us = 2.4 + div_up(groups, kCus) * (0.84 + H / 32 * c.cost / s * (1.0 + 0.44 * used));
            if (s > 1) us += 2.2 + 0.46e-6 * sizeof(float) * s * T * E;
            us = std::max(us, s > 1 ? 6.6 : 4.1);
            if (us < least) least = us, best = RouterChoice{c.kernel, c.bm, c.bn, s};
        });
    });
    return best;
}

// Every tiling at every number of rows of tiles that it may split, whatever the estimate says of it.
size_t most_router_workspace(int T, int H, int E, int parts) {
    int64_t most = 0;
    each_tiling(parts, [&](const Tiling& c) {
        if (!allowed(c, E)) return;
        const int across = div_up(E, c.bn);
        for (int m = 1; m <= div_up(T, c.bm) && m * across <= kCus; ++m)
            each_split(c, (int64_t)m * across, H, [&](int s) {
                if (s > 1) most = std::max(most, std::min((int64_t)s * std::min(m * c.bm, T) * E, kMostPartial));
            });
    });
    return (size_t)most * sizeof(float);
}

hipError_t launch_router_prepare(int H, int E, int weight_type, const void* w, uint8_t* w_tiled, hipStream_t stream) {
    const int64_t slots = (int64_t)((E + 15) / 16) * (H / 32) * 64;
    const dim3 grid((unsigned)((slots + kThreads - 1) / kThreads));
    if (weight_type == MOE_F32)
        hipLaunchKernelGGL(router_prepare_kernel<MOE_F32>, grid, dim3(kThreads), 0, stream, w, H, E, slots, w_tiled);
    else
        hipLaunchKernelGGL(router_prepare_kernel<MOE_BF16>, grid, dim3(kThreads), 0, stream, w, H, E, slots, w_tiled);
    return hipGetLastError();
}

namespace {
hipError_t launch_rows(const RouterArgs& a, RouterChoice c, hipStream_t stream) {
    const bool f32 = a.parts == 3;
    switch ((Kernel)c.kernel) {
        case kSmall: return f32 ? launch_small<3>(a, stream) : launch_small<1>(a, stream);
        case kTile32x64:
            return f32 ? launch_tile<Tile<32, 1, 8, 128, 3>>(a, c.splits, stream)
                       : launch_tile<Tile<32, 1, 8, 128, 1>>(a, c.splits, stream);
        case kTile32x128: return launch_tile<Tile<32, 2, 8, 128, 1>>(a, c.splits, stream);
        case kTile64x64:
            return f32 ? launch_tile<Tile<64, 1, 8, 128, 3>>(a, c.splits, stream)
                       : launch_tile<Tile<64, 1, 8, 128, 1>>(a, c.splits, stream);
        case kTile64x128:
            return f32 ? launch_tile<Tile<64, 2, 8, 64, 3>>(a, c.splits, stream)
                       : launch_tile<Tile<64, 2, 8, 128, 1>>(a, c.splits, stream);
        case kTile128x128: return launch_tile<Tile<128, 2, 8, 64, 3>>(a, c.splits, stream);
        case kTile128x192: return launch_tile<Tile<128, 3, 4, 128, 1>>(a, c.splits, stream);
        case kBig:
            if (a.x_stride >= kBigMaxStride) return launch_tile<Tile<128, 3, 4, 128, 1>>(a, 1, stream);
            hipLaunchKernelGGL(router_big_kernel, dim3((unsigned)div_up(a.T, Big::BM)), dim3(Big::WAVES * 64), 0, stream, a);
            return hipGetLastError();
        case kTile128x256: return launch_tile<Tile<128, 4, 4, 128, 1>>(a, c.splits, stream);
    }
    return hipErrorInvalidValue;
}
}  // namespace

hipError_t launch_router_logits(const RouterArgs& a, RouterChoice c, hipStream_t stream) {
    for (int64_t t = 0; t < a.T; t += kLaunchRows) {
        RouterArgs part = a;
        part.x += t * a.x_stride;
        part.logits += t * a.E;
        part.T = (int)std::min<int64_t>(a.T - t, kLaunchRows);
        const hipError_t e = launch_rows(part, c, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace moe
