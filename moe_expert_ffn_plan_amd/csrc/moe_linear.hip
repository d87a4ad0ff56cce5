// Dense product y = x W^T on the scaled matrix instructions: x E2M1 or E4M3, W E2M1, a UE8M0 scale per 32 columns.
#include "moe_internal.h"

#include <type_traits>
#include <utility>

namespace moe {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kStep = 128;       // columns of a K-step
constexpr int kBlockCodes = 2048, kBlockScales = 128;  // bytes of 32 weight rows in a K-step
constexpr int kNumXcd = 8;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}
__device__ __forceinline__ const uint8_t* uniform_ptr(const uint8_t* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<const uint8_t*>(((uint64_t)hi << 32) | lo);
}

// LDS DMA: lane l reads 16 (4) bytes at the wave-uniform base plus its own offset and writes them at LDS address
// lds + 16 l (4 l).  Issued from asm so that no wait for it is put in front of every LDS read.
__device__ __forceinline__ void dma16(uint32_t voff, const uint8_t* base, uint32_t lds) {
    asm volatile("global_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void dma4(uint32_t voff, const uint8_t* base, uint32_t lds) {
    asm volatile("global_load_lds_dword %0, %1" ::"v"(voff), "s"(base), "{m0}"(lds) : "memory");
}
// The lane, computed where it is used: what a tile derives from it once is then not kept in registers over its K-steps.
__device__ __forceinline__ int fresh_lane() {
    int l;
    asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
    return l;
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)p);
}
// At most N of this wave's DMA instructions stay in flight and its LDS reads are done; then all waves meet.
template <int N>
__device__ __forceinline__ void wait_and_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}
struct Args {
    const uint8_t* x;
    const uint8_t* sf;
    const uint8_t* w;
    const uint8_t* w_sf;
    uint16_t* y;
    float* partial;       // [splits][M][columns] where splits > 1
    int64_t y_stride;
    int64_t x_row;        // bytes of a row of codes
    // scales of x as words: row m of K-step kt at (m / 64) * sf_band + (m % 64) * sf_row + kt * sf_step
    int64_t sf_band;
    int sf_row, sf_step;
    int M, N, KT;
    bool wide;            // rows of y can be stored 8 outputs at a time
    bool stream;          // y is larger than the L2s together: its lines would only push out x's and the weights'
    int blocks;           // blocks of 32 weight rows
    int splits, per;      // K-steps of a split
    int mt, nt;           // tiles
};

__device__ __forceinline__ int64_t partial_columns(const Args& a) { return (int64_t)a.blocks * 32; }

// Two neighbouring outputs of a row.
__device__ __forceinline__ void store2(const Args& a, int row, int col, float v0, float v1) {
    uint16_t* out = a.y + (int64_t)row * a.y_stride + col;
    const uint32_t both = pack_bf16(v0, v1);
    if ((a.y_stride & 1) == 0 && col + 1 < a.N) {
        *reinterpret_cast<uint32_t*>(out) = both;
    } else {
        if (col < a.N) out[0] = (uint16_t)both;
        if (col + 1 < a.N) out[1] = (uint16_t)(both >> 16);
    }
}

// One tile of BM x BN outputs per workgroup, WM x WN waves.
//
// A K-step of 128 columns is a stage of a ring of NS in LDS, filled by DMA.  It is multiplied in two halves by
// V_MFMA_SCALE_F32_32X32X64: the hardware's two blocks of 32 columns are, in half s, the K-step's blocks s and 2 + s,
// so that lane l (row l % 32, q = l / 32) finds its two scales, of blocks 2q and 2q + 1, side by side in its row's word.
// An E2M1 lane holds the 32 columns of block 2q + s; an E4M3 lane 16 columns of each of the two blocks.  Rows of codes
// are 64 or 128 bytes with their 16-byte chunks permuted by the row (chunk ^ (row / 4) % 4, or ^ (row / 2) % 8): the 16
// lanes that LDS serves together (0-3, 12-15, 20-27 and so on) then read distinct banks of its 64.
//
// Half 1 of a stage is read while half 0 is multiplied, and half 0 of the next stage while half 1 is; the barrier that
// hands over a stage's buffer stands between the two.
//
// AK = 2: the rows of x come two K-steps at a time, into a ring of their own of two units.  Rows of 64 bytes are half a
// line each, and a request for half a line takes as long as one for a line (16384 x 7168 x 4096 E2M1: 237 us, 243 by one).
//
// Workgroups stay: each takes a run of tiles, whose outputs go through LDS to whole lines while the next tile's first stages
// load (237 us to 214).  Bound: 16384 x 7168 x 4096 E2M1 takes 205-224 us, 4300-4700 TFLOP/s of the 6960 that the
// instructions reach from registers, with the matrix cores busy 70% of the time at the clock that the load leaves; without
// DMA 190-200, without products 170-200.  E4M3 takes 312-346 (2800-3100 of 4310).  256 x 256 tiles, 64 x 128 to a wave,
// read least LDS for a product; 128 x 256 tiles, two to a CU, take 258, four waves 273.  128 x 128 tiles, two to a CU, fill
// the card where rows are fewer (2047 x 4064 x 1537 E4M3: 22 us to 32).
template <int FMT, int BM, int BN, int WM, int WN, int AK, int NS_>
struct Tile {
    static constexpr int W = WM * WN, THREADS = 64 * W, NS = NS_;
    static constexpr int KB = FMT == MOE_E2M1 ? 64 : 128;  // bytes of a row in a K-step
    static constexpr int RB = AK * KB;                     // and in what a DMA instruction loads
    static constexpr int CHUNKS = RB / 16;
    static constexpr int MI = BM / WM / 32, NI = BN / WN / 32;
    static constexpr int UNIT = BM * RB, UNITS = AK == 1 ? NS : 2;  // of x; behind them the stages of everything else
    static constexpr int B = 0, S = B + BN * 64, STAGE = S + (BM + BN) * 4, RING = UNITS * UNIT + NS * STAGE;
    static constexpr int OUT = 8 * (BN / WN) * 2, LDS = RING + W * OUT;  // of a wave: 8 rows of its outputs
    static constexpr int A_I = BM * RB / 1024, B_I = BN * 64 / 1024, S_I = (BM + BN) / 64;  // DMA instructions
    static constexpr int A_PW = (A_I + W - 1) / W, B_PW = (B_I + W - 1) / W, S_PW = (S_I + W - 1) / W;
    static constexpr int D = (AK == 1 ? A_PW : 0) + B_PW + S_PW;  // of a stage
    static __device__ __forceinline__ int permuted(int row) { return CHUNKS == 4 ? (row >> 2) & 3 : (row >> 1) & 7; }
    static_assert(CHUNKS == 4 || CHUNKS == 8, "rows of 64 or 128 bytes");
    static_assert(BM % 64 == 0 && BN % 64 == 0 && NI % 2 == 0 && NS >= 2 && (NS - 1) * D < 63, "tile");
    static_assert(W * 64 / CHUNKS % 16 == 0 && A_I % W == 0, "rows of a wave's instructions");
};

template <int FMT>
struct Frag {
    typedef v4i type;
};
template <>
struct Frag<MOE_E4M3> {
    typedef v8i type;
};

template <int FMT, int H>
__device__ __forceinline__ v16f mfma(const typename Frag<FMT>::type& a, const v4i& b, const v16f& c, int sa, int sb) {
    const v8i b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
    if constexpr (FMT == MOE_E2M1) {
        const v8i a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, H, sa, H, sb);
    } else {
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b8, c, 0, 4, H, sa, H, sb);
    }
}

template <class F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}

template <int FMT, int BM, int BN, int WM, int WN, int AK, int NS, int OCC>
__global__ __launch_bounds__(64 * WM * WN, OCC) void tile_kernel(Args g) {
    using T = Tile<FMT, BM, BN, WM, WN, AK, NS>;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS];
    auto unit_of = [&](int u) { return smem + u % T::UNITS * T::UNIT; };
    auto stage_of = [&](int t) { return smem + T::UNITS * T::UNIT + t % NS * T::STAGE; };

    // every XCD takes a contiguous run of tiles, in columns of 8 tile rows, so that what runs together shares
    // its rows of x and its weights in the XCD's L2; a workgroup takes every (workgroups of an XCD)-th of its run
    const int per_split = g.mt * g.nt, tiles = per_split * g.splits;
    const int share = (tiles + kNumXcd - 1) / kNumXcd, xcd = blockIdx.x % kNumXcd;
    const int last = min((xcd + 1) * share, tiles), stride = gridDim.x / kNumXcd;
    int id = xcd * share + blockIdx.x / kNumXcd;
    if (id >= last) return;

    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);

    // ---- DMA sources of a tile
    int m0, n0, z, k0, n;  // its first row, output, split, K-step, and its K-steps
    const uint8_t* x;
    // the rows of a wave's instructions lie W * 64 / CHUNKS apart, a multiple of the permutation's 16
    const uint32_t chunk = ((lane % T::CHUNKS) ^ T::permuted(w * (64 / T::CHUNKS) + lane / T::CHUNKS)) * 16;
    uint32_t a_row[T::A_PW], s_off[T::S_PW], s_step[T::S_PW];
    const uint8_t* b_src[T::B_PW];
    const uint8_t* s_src[T::S_PW];
    auto take = [&](int tile) {
        const int lane = fresh_lane();
        z = tile / per_split;
        const int in = tile % per_split;
        const int band = in / (8 * g.nt), rows = min(8, g.mt - band * 8), at = in - band * 8 * g.nt;
        m0 = (band * 8 + at % rows) * BM;
        n0 = at / rows * BN;
        k0 = z * g.per;
        n = min(g.per, g.KT - k0);
        x = uniform_ptr(g.x + (int64_t)m0 * g.x_row);
#pragma unroll
        for (int i = 0; i < T::A_PW; ++i) {
            const int row = (i * T::W + w) % T::A_I * (64 / T::CHUNKS) + lane / T::CHUNKS;
            a_row[i] = (uint32_t)min(row, g.M - 1 - m0) * (uint32_t)g.x_row;
        }
        const int nb0 = n0 / 32;
#pragma unroll
        for (int i = 0; i < T::B_PW; ++i) {
            const int blk = (i * T::W + w) % T::B_I;
            b_src[i] = uniform_ptr(g.w + (int64_t)min(nb0 + blk / 2, g.blocks - 1) * g.KT * kBlockCodes + (blk & 1) * 1024);
        }
        // a wave's scales of row r of its blocks of 32 lie side by side: word (part * 32 + r) * blocks + i is that of row
        // part * 32 * blocks + 32 i + r
#pragma unroll
        for (int i = 0; i < T::S_PW; ++i) {
            const int idx = (i * T::W + w) % T::S_I;
            if (idx < BM / 64) {  // rows of x
                const int word = idx * 64 + lane, at = word / T::MI;
                const int row = at / 32 * (32 * T::MI) + word % T::MI * 32 + at % 32;
                const int m = min(row, g.M - 1 - m0);
                s_src[i] = uniform_ptr(g.sf + m0 / 64 * g.sf_band);
                s_step[i] = g.sf_step;
                s_off[i] = (uint32_t)(m / 64) * (uint32_t)g.sf_band + (uint32_t)(m % 64) * (uint32_t)g.sf_row;
            } else {  // weight rows
                const int word = (idx - BM / 64) * 64 + lane, at = word / T::NI;
                const int blk = at / 32 * T::NI + word % T::NI;
                s_src[i] = uniform_ptr(g.w_sf + (int64_t)nb0 * g.KT * kBlockScales);
                s_step[i] = kBlockScales;
                s_off[i] = (uint32_t)min(blk, g.blocks - 1 - nb0) * (uint32_t)g.KT * kBlockScales + (uint32_t)(at % 32) * 4;
            }
        }
    };
    // DMA instruction i of unit u of x: K-steps k0 + AK u and on.  Columns past the last are those of the row's last chunk:
    // the weights there are 0.
    auto issue_a = [&](int i, int u) {
        const uint32_t at = (uint32_t)(k0 + u * AK) * T::KB + chunk;
        dma16(a_row[i] + min(at, (uint32_t)g.x_row - 16), x, lds_addr(unit_of(u) + (i * T::W + w) % T::A_I * 1024));
    };
    // of stage t, in place of stage `to`
    auto issue1 = [&](int i, int to, int t) {
        uint8_t* st = stage_of(to);
        const int kt = k0 + t;
        if constexpr (AK == 1) {
            if (i < T::A_PW) {
                const uint32_t at = (uint32_t)kt * T::KB + chunk;
                dma16(a_row[i] + min(at, (uint32_t)g.x_row - 16), x, lds_addr(unit_of(to) + (i * T::W + w) % T::A_I * 1024));
                return;
            }
            i -= T::A_PW;
        }
        if (i < T::B_PW) {
            dma16((uint32_t)lane * 16, b_src[i] + (int64_t)kt * kBlockCodes, lds_addr(st + T::B + (i * T::W + w) % T::B_I * 1024));
        } else {
            i -= T::B_PW;
            dma4(s_off[i], s_src[i] + (int64_t)kt * s_step[i], lds_addr(st + T::S + (i * T::W + w) % T::S_I * 256));
        }
    };

    // ---- fragments
    const int r = lane & 31, q = lane >> 5, rsw = T::permuted(r), bsw = (r >> 2) & 3;
    const int wm = w / WN, wn = w % WN, wm0 = wm * (BM / WM), wn0 = wn * (BN / WN);
    typedef typename Frag<FMT>::type fa;
    struct Half {
        fa a[T::MI];
        v4i b[T::NI];
    };
    // fragment i of half h of K-step t, in the order in which they are multiplied
    auto read1 = [&](int i, Half& f, int t, int h) {
        if (i == 0 || i > T::NI) {
            i = i == 0 ? 0 : i - T::NI;
            const uint8_t* row = unit_of(t / AK) + (wm0 + i * 32 + r) * T::RB;
            if constexpr (FMT == MOE_E2M1) {
                f.a[i] = *reinterpret_cast<const v4i*>(row + (((t % AK * 4 + 2 * q + h) ^ rsw) << 4));
            } else {
                const v4i lo = *reinterpret_cast<const v4i*>(row + (((2 * h + q) ^ rsw) << 4));
                const v4i hi = *reinterpret_cast<const v4i*>(row + (((4 + 2 * h + q) ^ rsw) << 4));
                f.a[i] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            }
        } else {
            i -= 1;
            f.b[i] = *reinterpret_cast<const v4i*>(stage_of(t) + T::B + (wn0 + i * 32 + r) * 64 + (((2 * q + h) ^ bsw) << 4));
        }
    };
    struct Scales {
        int a[T::MI], b[T::NI];
    };
    auto read_scales = [&](Scales& f, int t) {
        const uint8_t* st = stage_of(t);
        typedef uint32_t va __attribute__((ext_vector_type(T::MI)));
        typedef uint32_t vb __attribute__((ext_vector_type(T::NI)));
        const va sa = *reinterpret_cast<const va*>(st + T::S + (wm * 32 + r) * T::MI * 4);
        const vb sb = *reinterpret_cast<const vb*>(st + T::S + BM * 4 + (wn * 32 + r) * T::NI * 4);
#pragma unroll
        for (int i = 0; i < T::MI; ++i) f.a[i] = (int)(sa[i] >> (16 * q));
#pragma unroll
        for (int i = 0; i < T::NI; ++i) f.b[i] = (int)(sb[i] >> (16 * q));
    };

    v16f acc[T::MI][T::NI];
    constexpr int FRAGS = T::MI + T::NI, SLOTS = T::MI * T::NI, PER = (FRAGS + SLOTS - 1) / SLOTS;
    Half f0, f1;
    Scales sc, sn;
    // K-step t.  The DMA of stage t + NS begins behind the barrier that frees its buffer (parts 0 .. D1 - 1, if `begin`)
    // and goes on in front of the next (`finish`, of stage t + NS - 1): in one burst the waves wait for each other's
    // requests.  With AK = 2 that of a unit of x does so behind an odd K-step (`begin_a`, `finish_a`).  flight: this wave's
    // DMA instructions behind those of K-step t + 1.  The order is pinned: reads and DMA stand between the products, so
    // that the matrix core always has the next one.
    constexpr int D1 = T::D / 2, A1 = T::A_PW / 2;
    auto dma_slot = [](int i, int count) { return (2 * i + 1) * SLOTS / (2 * count); };
    auto step = [&](int t, auto finish, auto begin, auto finish_a, auto begin_a, auto flight) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < SLOTS; ++k) {
            const int i = k / T::NI, j = k % T::NI;
            acc[i][j] = mfma<FMT, 0>(f0.a[i], f0.b[j], acc[i][j], sc.a[i], sc.b[j]);
#pragma unroll
            for (int h = k * PER; h < min((k + 1) * PER, FRAGS); ++h) read1(h, f1, t, 1);
            constexpr int MA = decltype(finish_a)::value ? T::A_PW - A1 : 0, MB = decltype(finish)::value ? T::D - D1 : 0;
#pragma unroll
            for (int h = 0; h < MA + MB; ++h)
                if (dma_slot(h, MA + MB) == k) {
                    if (h < MA) issue_a(A1 + h, t / 2 + 1);
                    else issue1(D1 + h - MA, t + NS - 1, min(t + NS - 1, n - 1));
                }
            __builtin_amdgcn_sched_barrier(0);
        }
        wait_and_barrier<decltype(flight)::value>();  // K-step t + 1 is there, K-step t read
#pragma unroll
        for (int k = 0; k < SLOTS; ++k) {
            const int i = k / T::NI, j = k % T::NI;
            acc[i][j] = mfma<FMT, 1>(f1.a[i], f1.b[j], acc[i][j], sc.a[i], sc.b[j]);
#pragma unroll
            for (int h = k * PER; h < min((k + 1) * PER, FRAGS); ++h) read1(h, f0, t + 1, 0);
            if (k == SLOTS / 2) read_scales(sn, t + 1);
            constexpr int MA = decltype(begin_a)::value ? A1 : 0, MB = decltype(begin)::value ? D1 : 0;
#pragma unroll
            for (int h = 0; h < MA + MB; ++h)
                if (dma_slot(h, MA + MB) == k) {
                    if (h < MA) issue_a(h, (t + 3) / 2);
                    else issue1(h - MA, t, t + NS);
                }
            __builtin_amdgcn_sched_barrier(0);
        }
        sc = sn;
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    // the first stages of a tile
    auto fill = [&]() {
    if constexpr (AK == 1) {
        // a split of fewer than NS K-steps fills the ring with its last one
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
            for (int i = 0; i < (u < NS - 1 ? T::D : D1); ++i) issue1(i, u, min(u, n - 1));
    } else {  // in the order of the steps that would come before the first: of each stage, and of unit 0 with stage 1
#pragma unroll
        for (int i = 0; i < T::D; ++i) issue1(i, 0, 0);
#pragma unroll
        for (int i = 0; i < T::A_PW; ++i) issue_a(i, 0);
#pragma unroll
        for (int i = 0; i < T::D; ++i) issue1(i, 1, 1);
#pragma unroll
        for (int i = 0; i < T::D; ++i) issue1(i, 2, 2);
#pragma unroll
        for (int i = 0; i < A1; ++i) issue_a(i, 1);
#pragma unroll
        for (int i = 0; i < D1; ++i) issue1(i, 3, 3);
    }
    };
    take(id);
    fill();
    for (;;) {
    wait_and_barrier<AK == 1 ? (NS - 2) * T::D + D1 : 2 * T::D + A1 + D1>();
#pragma unroll
    for (int i = 0; i < T::MI; ++i)
#pragma unroll
        for (int j = 0; j < T::NI; ++j) acc[i][j] = v16f{};
    int t = 0;
#pragma unroll
    for (int i = 0; i < FRAGS; ++i) read1(i, f0, 0, 0);
    read_scales(sc, 0);
    if constexpr (AK == 1) {
        for (; t < n - NS; ++t) step(t, yes, yes, no, no, std::integral_constant<int, (NS - 2) * T::D>{});
        step(t++, yes, no, no, no, std::integral_constant<int, (NS - 2) * T::D>{});
        auto tail = [&](auto i) {
            constexpr int later = NS - 2 - decltype(i)::value;
            if (t < n) step(t++, no, no, no, no, std::integral_constant<int, (later > 0 ? later : 0) * T::D>{});
        };
        each_of([&](auto i) { tail(std::integral_constant<int, decltype(i)::value + 1>{}); },
                std::make_integer_sequence<int, NS - 1>{});
    } else {
        static_assert(AK == 1 || NS == 4, "what is in flight");
        // At the barrier of an even step stages t + 2 and t + 3 are in flight and the unit that was begun behind t - 1; of an
        // odd one, whose next step needs that unit, what followed it: the rest of stage t + 2, and stage t + 3.
        constexpr int EVEN = 2 * T::D + T::A_PW, ODD = 2 * T::D - D1;
        for (; t + 1 + NS < n;) {
            step(t++, yes, yes, yes, no, std::integral_constant<int, EVEN>{});
            step(t++, yes, yes, no, yes, std::integral_constant<int, ODD>{});
        }
        // the last NS or NS + 1, of which the one behind the NS has not been begun
        const int rest = n - t;
#pragma unroll
        for (int i = A1; i < T::A_PW; ++i) issue_a(i, t / 2 + 1);
#pragma unroll
        for (int i = D1; i < T::D; ++i) issue1(i, t + NS - 1, t + NS - 1);
        for (; t < n; ++t) {
            const int left = n - t;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < SLOTS; ++k) {
                const int i = k / T::NI, j = k % T::NI;
                acc[i][j] = mfma<FMT, 0>(f0.a[i], f0.b[j], acc[i][j], sc.a[i], sc.b[j]);
#pragma unroll
                for (int h = k * PER; h < min((k + 1) * PER, FRAGS); ++h) read1(h, f1, t, 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (left == rest) wait_and_barrier<EVEN>();
            else if (left == NS && rest == NS + 1) wait_and_barrier<ODD>();
            else if (left == NS - 1 && rest == NS) wait_and_barrier<T::D - D1>();
            else if (left == 3 && rest == NS + 1) wait_and_barrier<T::D + T::A_PW>();
            else wait_and_barrier<0>();
            if (left == NS + 1) {
#pragma unroll
                for (int i = 0; i < T::D; ++i) issue1(i, t, n - 1);
            }
            if (left == NS && rest == NS + 1) {
#pragma unroll
                for (int i = 0; i < T::A_PW; ++i) issue_a(i, (n - 1) / 2);
            }
#pragma unroll
            for (int k = 0; k < SLOTS; ++k) {
                const int i = k / T::NI, j = k % T::NI;
                acc[i][j] = mfma<FMT, 1>(f1.a[i], f1.b[j], acc[i][j], sc.a[i], sc.b[j]);
#pragma unroll
                for (int h = k * PER; h < min((k + 1) * PER, FRAGS); ++h) read1(h, f0, t + 1, 0);
                if (k == SLOTS / 2) read_scales(sn, t + 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            sc = sn;
        }
    }

    // Nothing is on its way to LDS any more (a split of fewer than NS K-steps filled the ring all the same), and no wave
    // reads it.  The next tile's first stages are loaded while this one's outputs are stored.
    wait_and_barrier<0>();
    const int om = m0 + wm0, on = n0 + wn0;
    float* part = g.partial + (int64_t)z * g.M * partial_columns(g);
    id += stride;
    if (id < last) {
        take(id);
        fill();
    }

    // ---- outputs: weight rows are laid so that lane r of blocks 2b and 2b + 1 holds outputs 2r and 2r + 1 of their 64
    const int l = fresh_lane(), c = 2 * (l & 31), p = l >> 5;
    if (g.splits > 1) {
#pragma unroll
        for (int i = 0; i < T::MI; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int row = om + i * 32 + 8 * (e / 4) + 4 * p + e % 4;
#pragma unroll
                for (int j = 0; j < T::NI; j += 2) {
                    const int col = on + j * 32 + c;
                    if (row < g.M && col < partial_columns(g))
                        *reinterpret_cast<f32x2*>(part + (int64_t)row * partial_columns(g) + col) =
                            f32x2{acc[i][j][e], acc[i][j + 1][e]};
                }
            }
    } else if (g.wide) {
        auto store = [&](auto stream) {
        // 8 rows at a time through LDS, where each wave has a place of its own, so that a store is whole lines
        constexpr int COLS = BN / WN, LANES = COLS / 8;  // lanes of a row
        uint8_t* place = smem + T::RING + w * T::OUT;
#pragma unroll
        for (int i = 0; i < T::MI; ++i)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int j = 0; j < T::NI; j += 2)
                        *reinterpret_cast<uint32_t*>(place + ((4 * p + k) * COLS + j * 32 + c) * 2) =
                            pack_bf16(acc[i][j][e + k], acc[i][j + 1][e + k]);
                wave_exchange();
#pragma unroll
                for (int h = 0; h < 8 * LANES / 64; ++h) {
                    const int at = h * 64 + l;
                    const v4i v = *reinterpret_cast<const v4i*>(place + at * 16);
                    const int row = om + i * 32 + 2 * e + at / LANES, col = on + at % LANES * 8;
                    if (row < g.M && col < g.N) {
                        v4i* to = reinterpret_cast<v4i*>(g.y + (int64_t)row * g.y_stride + col);
                        if constexpr (decltype(stream)::value) __builtin_nontemporal_store(v, to);
                        else *to = v;
                    }
                }
                wave_exchange();
            }
        };
        if (g.stream) store(yes);
        else store(no);
    } else {
#pragma unroll
        for (int i = 0; i < T::MI; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int row = om + i * 32 + 8 * (e / 4) + 4 * p + e % 4;
#pragma unroll
                for (int j = 0; j < T::NI; j += 2)
                    if (row < g.M) store2(g, row, on + j * 32 + c, acc[i][j][e], acc[i][j + 1][e]);
            }
    }
    if (id >= last) break;
    }
}

// Few rows of x: what counts is how the weights stream in.  A workgroup takes a block of 32 weight rows over all columns,
// its W waves U K-steps each in turn.  The weights go straight from memory to the matrix instructions' registers (no two
// waves read the same ones, so LDS would only be a detour).  x goes through LDS, where each wave has a place of its own and
// needs no barrier: lanes that load neighbouring chunks of few rows touch few lines, lanes that load what they multiply
// touch one each.  The waves' sums are added through LDS, in the waves' order.
// Bound by the launch and by the weights' latency: 1 x 7168 x 4096 E4M3 takes 4.9 us, 32 rows 6.3 to 7.3, 64 8.7 to 9.2, 128 (two
// groups, E2M1) 8.9 to 9.7; the same in tiles 11.8 to 14.8.
template <int FMT, int ROWS, int W, int U>
struct Few {
    static constexpr int RB = FMT == MOE_E2M1 ? 64 : 128, BYTES = U * RB, CHUNKS = BYTES / 16;  // of a row in a turn
    static constexpr int MI = (ROWS + 31) / 32, PER = 64 / CHUNKS;                              // rows of a DMA instruction
    static constexpr int PLACE = ROWS * BYTES, SUMS = MI * 16 * 64 * 4;                         // of a wave
    static constexpr int LDS = W * (PLACE > SUMS ? PLACE : SUMS);
    static_assert(CHUNKS >= 16 && CHUNKS <= 64 && LDS <= 160 * 1024, "place of a wave");
};

template <int FMT, int ROWS, int W, int U>
__global__ __launch_bounds__(64 * W) void few_kernel(Args g) {
    using F = Few<FMT, ROWS, W, U>;
    typedef typename Frag<FMT>::type fa;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[F::LDS];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, q = lane >> 5, b = blockIdx.x;
    const int m0 = blockIdx.y * ROWS, rows = min(g.M - m0, ROWS);
    const uint8_t* x = uniform_ptr(g.x + (int64_t)m0 * g.x_row);
    uint8_t* place = smem + w * F::PLACE;
    const int row_bytes = (int)g.x_row, blocks = g.sf_row;  // of scales: bytes, one for 32 columns
    const uint8_t* code = g.w + (int64_t)b * g.KT * kBlockCodes + r * 64;
    const uint8_t* scale = g.w_sf + (int64_t)b * g.KT * kBlockScales + r * 4;
    const int c0 = ((2 * q) ^ ((r >> 2) & 3)) * 16;  // of half 0; half 1 is its neighbour
    v16f acc[F::MI];
#pragma unroll
    for (int i = 0; i < F::MI; ++i) acc[i] = v16f{};
    for (int kt0 = w * U; kt0 < g.KT; kt0 += W * U) {
        // columns past the last are those of the row's last chunk, and its last scale: the weights there are 0
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the last turn's reads are done
#pragma unroll
        for (int i = 0; i < ROWS / F::PER; ++i) {
            if (i * F::PER >= rows) break;
            const int row = i * F::PER + lane / F::CHUNKS;
            const int chunk = (lane % F::CHUNKS) ^ (row & 15);
            const uint32_t at = (uint32_t)min(row, rows - 1) * (uint32_t)row_bytes +
                                (uint32_t)min(kt0 * F::RB + chunk * 16, row_bytes - 16);
            dma16(at, x, lds_addr(place + i * 1024));
        }
        v4i wc[U][2];
        uint32_t ws[U], xs[F::MI][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kt = min(kt0 + u, g.KT - 1);
            const uint8_t* at = code + (int64_t)kt * kBlockCodes;
            wc[u][0] = *reinterpret_cast<const v4i*>(at + c0);
            wc[u][1] = *reinterpret_cast<const v4i*>(at + (c0 ^ 16));
            ws[u] = *reinterpret_cast<const uint32_t*>(scale + (int64_t)kt * kBlockScales);
        }
#pragma unroll
        for (int i = 0; i < F::MI; ++i) {  // a turn's scales of a row lie side by side
            const uint8_t* sf = g.sf + (int64_t)(m0 + min(i * 32 + r, rows - 1)) * blocks + kt0 * 4;
            if ((kt0 + U) * 4 <= blocks) {
                __builtin_memcpy(&xs[i][0], sf, U * 4);
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    xs[i][u] = 0;
                    for (int k = 0; k < 4; ++k)
                        if ((kt0 + u) * 4 + k < blocks) xs[i][u] |= (uint32_t)sf[u * 4 + k] << (8 * k);
                }
            }
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (kt0 + u >= g.KT) break;
            const int sb = (int)(ws[u] >> (16 * q));
#pragma unroll
            for (int i = 0; i < F::MI; ++i) {
                const uint8_t* row = place + (ROWS < 32 ? r % ROWS : i * 32 + r) * F::BYTES;
                const int sa = (int)(xs[i][u] >> (16 * q));
                auto chunk = [&](int c) { return *reinterpret_cast<const v4i*>(row + (((u * (F::RB / 16) + c) ^ (r & 15)) << 4)); };
                fa a0, a1;
                if constexpr (FMT == MOE_E2M1) {
                    a0 = chunk(2 * q);
                    a1 = chunk(2 * q + 1);
                } else {
                    const v4i c00 = chunk(q), c01 = chunk(4 + q), c10 = chunk(2 + q), c11 = chunk(6 + q);
                    a0 = v8i{c00[0], c00[1], c00[2], c00[3], c01[0], c01[1], c01[2], c01[3]};
                    a1 = v8i{c10[0], c10[1], c10[2], c10[3], c11[0], c11[1], c11[2], c11[3]};
                }
                acc[i] = mfma<FMT, 0>(a0, wc[u][0], acc[i], sa, sb);
                acc[i] = mfma<FMT, 1>(a1, wc[u][1], acc[i], sa, sb);
            }
        }
    }
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);  // [W][MI * 16][64]
#pragma unroll
    for (int i = 0; i < F::MI; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (i * 32 + 8 * (e / 4) < rows) sums[((w * F::MI + i) * 16 + e) * 64 + lane] = acc[i][e];
    __syncthreads();
    for (int o = threadIdx.x; o < F::MI * 1024; o += 64 * W) {
        const int at = o & 63, e = o / 64 % 16, i = o / 1024;
        const int row = i * 32 + 8 * (e / 4) + 4 * (at >> 5) + e % 4;
        const int col = (b >> 1) * 64 + 2 * (at & 31) + (b & 1);
        if (row >= rows || col >= g.N) continue;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) v += sums[((k * F::MI + i) * 16 + e) * 64 + at];
        g.y[(int64_t)(m0 + row) * g.y_stride + col] = (uint16_t)pack_bf16(v, v);
    }
}

constexpr int kThreads = 256;

// The splits' sums, in their order.
__global__ __launch_bounds__(kThreads) void join_kernel(Args g) {
    const int64_t columns = partial_columns(g), at = (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x) * 4;
    if (at >= (int64_t)g.M * columns) return;
    v4f v = {0.f, 0.f, 0.f, 0.f};
    for (int z = 0; z < g.splits; ++z) v += *reinterpret_cast<const v4f*>(g.partial + (int64_t)z * g.M * columns + at);
    const int row = (int)(at / columns), col = (int)(at % columns);
    store2(g, row, col, v[0], v[1]);
    store2(g, row, col + 2, v[2], v[3]);
}

// Scales of x by K-step, [M/64][KT][64 rows][4 B], zeros behind the last column: what a tile loads of a K-step is then
// whole lines.  A workgroup turns 64 rows of kTurn K-steps in LDS, so that it reads along rows and writes along K-steps.
constexpr int kTurn = 8;
__global__ __launch_bounds__(kThreads) void tile_scales_kernel(const uint8_t* sf, int M, int blocks, int KT, uint32_t* out) {
    __shared__ uint32_t words[kTurn][72];  // the 8 K-steps of 8 rows, which are written together, to 64 banks
    const int chunks = (KT + kTurn - 1) / kTurn;
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, band = block / chunks;
    const int kt0 = (int)(block % chunks) * kTurn;
    if (band * 64 >= M) return;
    const int kt = kt0 + threadIdx.x % kTurn;
#pragma unroll
    for (int i = 0; i < 64; i += kThreads / kTurn) {
        const int in = i + threadIdx.x / kTurn;
        const int64_t row = band * 64 + in;
        uint32_t v = 0;
        if (row < M && kt < KT) {
            const uint8_t* at = sf + row * blocks + kt * 4;
            if (blocks % 4 == 0) {
                v = *reinterpret_cast<const uint32_t*>(at);
            } else {
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (kt * 4 + b < blocks) v |= (uint32_t)at[b] << (8 * b);
            }
        }
        words[threadIdx.x % kTurn][in] = v;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTurn; i += kThreads / 64) {
        const int step = i + threadIdx.x / 64;
        if (kt0 + step < KT) out[(band * KT + kt0 + step) * 64 + threadIdx.x % 64] = words[step][threadIdx.x % 64];
    }
}

template <int FMT, int BM, int BN, int WM, int WN, int AK, int NS, int OCC>
void go(const Args& g, hipStream_t stream) {
    const int tiles = g.mt * g.nt * g.splits, share = (tiles + kNumXcd - 1) / kNumXcd;
    constexpr int PER_CU = 160 * 1024 / Tile<FMT, BM, BN, WM, WN, AK, NS>::LDS;
    const int per_xcd = std::min(share, std::max(1, cu_count() / kNumXcd * PER_CU));
    hipLaunchKernelGGL((tile_kernel<FMT, BM, BN, WM, WN, AK, NS, OCC>), dim3((unsigned)(per_xcd * kNumXcd)), dim3(64 * WM * WN), 0,
                       stream, g);
}

template <int FMT, int ROWS, int W, int U>
void few(const Args& g, hipStream_t stream) {
    hipLaunchKernelGGL((few_kernel<FMT, ROWS, W, U>), dim3((unsigned)g.blocks, (unsigned)((g.M + ROWS - 1) / ROWS)),
                       dim3(64 * W), 0, stream, g);
}

}  // namespace

constexpr int kFewRows = 64, kSomeRows = 128;
constexpr int kLongSteps = 5;    // K-steps that the ring of two units of x needs; shorter tiles load it by one
constexpr int kFillTiles = 256;  // a workgroup for every compute unit
constexpr int kMostSplits = 16, kLeastSteps = 4;

static size_t laid_out_bytes(int M, int KT) { return ((size_t)M + 63) / 64 * KT * 256; }  // of x's scales by K-step

// The kernel with the least estimated time, in microseconds (measured at 2048 .. 16384 rows, 2016 .. 7168 columns and 512
// .. 7168 outputs, most within 15%, and taken from 65 rows up for any size): a K-step of a 256 x 256 tile takes 0.8 (E2M1) or 1.3 (E4M3), one of a 128 x 128 tile
// 0.27 or 0.4, or 0.36 or 0.42 for each of two that share a compute unit; to lay out the scales takes 4, to join splits 4 and their
// partial sums' way to memory and back.
MxLinearChoice choose_mx_linear(int M, int N, int K, int format) {
    MxLinearChoice c{};
    const int KT = mx_steps(K);
    const bool four = format == MOE_E2M1;
    c.splits = 1;
    const int64_t groups = ((int64_t)M + 63) / 64, blocks = mx_column_blocks(N);
    // up to 64 rows (64 x 7168 x 4096: 8.7 us, 12.3 in tiles), or 128 where all workgroups run at once (128 rows: 8.9, 14.8)
    if (M <= kFewRows || (M <= kSomeRows && groups * blocks <= kFillTiles)) {
        c.kernel = 2;
        c.tokens = M <= 32 ? 32 : 64;
        c.columns = 32;
        return c;
    }
    const int64_t big = (((int64_t)M + 255) / 256) * (((int64_t)N + 255) / 256);
    const int64_t small = (((int64_t)M + 127) / 128) * (((int64_t)N + 127) / 128);
    const double lay_out = K % kStep != 0 ? 4.0 : 0.0;
    double best = (double)((big + kFillTiles - 1) / kFillTiles) * (KT * (four ? 0.8 : 1.3) + 5.0) + 9.0;
    c.tokens = c.columns = 256;
    for (int splits = 1; splits <= kMostSplits; splits *= 2) {
        const int64_t tiles = small * splits;
        if (splits > 1 && (KT / splits < kLeastSteps || small >= kFillTiles || tiles > 2 * kFillTiles)) break;
        const double at_once = tiles <= kFillTiles ? 1.0 : 2.0 * (double)((tiles + 2 * kFillTiles - 1) / (2 * kFillTiles));
        const double step = at_once > 1.0 ? (four ? 0.36 : 0.42) : (four ? 0.27 : 0.4);
        double us = at_once * ((KT + splits - 1) / splits) * step + 4.0 + lay_out;
        if (splits > 1) us += 4.0 + (double)splits * M * N * 8.0 / 6e6;
        if (us >= best) continue;
        best = us;
        c.kernel = 1;
        c.tokens = c.columns = 128;
        c.splits = splits;
    }
    c.splits = (KT + c.split_steps(KT) - 1) / c.split_steps(KT);  // none without a K-step
    // A K-step's word of a row is a line of its own, so large tiles want them laid out; and words start at multiples of 4.
    c.tile_scales = K % kStep != 0 || c.kernel == 0;
    c.scale_bytes = c.tile_scales ? laid_out_bytes(M, KT) : 0;
    c.partial_bytes = c.splits > 1 ? (size_t)c.splits * M * mx_column_blocks(N) * 32 * 4 : 0;
    return c;
}

size_t most_mx_linear_workspace(int M, int N, int K, int format) {
    // Partial sums are had by fewer than kFillTiles tile rows alone: those batches are asked one by one.  Larger ones take
    // laid out scales or nothing, now this and now that as the tokens grow, and no more than the scales of M tokens.
    const int asked = std::min(M, kFillTiles * 128);
    size_t most = M > asked ? laid_out_bytes(M, mx_steps(K)) : 0;
    for (int m = asked; m > 0; --m) most = std::max(most, choose_mx_linear(m, N, K, format).workspace_bytes());
    return most;
}

hipError_t launch_mx_linear(const MxLinearArgs& a, const MxLinearChoice& c, hipStream_t stream) {
    Args g{};
    g.x = a.x;
    g.w = a.w;
    g.y = a.y;
    g.y_stride = a.y_stride;
    g.M = a.M;
    g.N = a.N;
    g.KT = mx_steps(a.K);
    g.blocks = (int)mx_column_blocks(a.N);
    g.w_sf = a.w + (int64_t)g.blocks * g.KT * kBlockCodes;
    const int per16 = a.format == MOE_E2M1 ? 2 : 1;  // codes of a byte
    g.x_row = a.K / per16;
    g.sf = a.x_sf;
    g.sf_band = (int64_t)a.K / 32 * 64;
    g.sf_row = a.K / 32;
    g.sf_step = 4;
    g.partial = reinterpret_cast<float*>(a.ws + c.scale_bytes);
    if (c.tile_scales) {
        g.sf = a.ws;
        g.sf_band = (int64_t)g.KT * 256;
        g.sf_row = 4;
        g.sf_step = 256;
        const int64_t turns = ((int64_t)a.M + 63) / 64 * ((g.KT + kTurn - 1) / kTurn);
        hipLaunchKernelGGL(tile_scales_kernel, wide_grid(turns), dim3(kThreads), 0, stream, a.x_sf, a.M, a.K / 32, g.KT,
                           reinterpret_cast<uint32_t*>(a.ws));
    }
    g.splits = c.splits;
    g.per = c.split_steps(g.KT);
    g.wide = a.N % 8 == 0 && a.y_stride % 8 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
    g.stream = (int64_t)a.M * a.N * 2 > 32ll << 20;
    g.mt = (a.M + c.tokens - 1) / c.tokens;
    g.nt = (a.N + c.columns - 1) / c.columns;
    if (c.kernel == 2) {
        if (a.format == MOE_E2M1) {
            if (a.M <= 32) few<MOE_E2M1, 32, 16, 4>(g, stream);
            else few<MOE_E2M1, 64, 8, 4>(g, stream);
        } else {
            if (a.M <= 16) few<MOE_E4M3, 16, 16, 4>(g, stream);
            else if (a.M <= 32) few<MOE_E4M3, 32, 16, 2>(g, stream);
            else few<MOE_E4M3, 64, 8, 2>(g, stream);
        }
    } else if (c.kernel == 0) {
        if (a.format == MOE_E4M3) go<MOE_E4M3, 256, 256, 2, 4, 1, 3, 2>(g, stream);
        else if (g.KT >= kLongSteps) go<MOE_E2M1, 256, 256, 2, 4, 2, 4, 2>(g, stream);
        else go<MOE_E2M1, 256, 256, 2, 4, 1, 4, 2>(g, stream);
    } else {
        if (a.format == MOE_E2M1) go<MOE_E2M1, 128, 128, 2, 2, 1, 4, 2>(g, stream);
        else go<MOE_E4M3, 128, 128, 2, 2, 1, 3, 2>(g, stream);
    }
    if (g.splits > 1)
        hipLaunchKernelGGL(join_kernel, wide_grid(((int64_t)a.M * (g.blocks * 32) / 4 + kThreads - 1) / kThreads),
                           dim3(kThreads), 0, stream, g);
    return hipGetLastError();
}

}  // namespace moe
