// Balance of the experts' load over sequences of rows, and the gradient of its loss and of the gate's weights.
//
// Both read a row of logits once.  A row is held by L neighbouring lanes, V values each: in runs of 4 where the rows
// allow vector loads (value i of lane l is expert 4 (l + L (i / 4)) + i % 4), else l + L i.
#include "moe_internal.h"

#include <type_traits>

namespace moe {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// ---- reductions over each L neighbouring lanes, the result in all of them
struct Sum {
    static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
struct IntSum {  // of ints in their bits
    static __device__ __forceinline__ float of(float a, float b) { return __int_as_float(__float_as_int(a) + __float_as_int(b)); }
};
struct Max {
    static __device__ __forceinline__ float of(float a, float b);
};
template <class Op, int CTRL>
__device__ __forceinline__ float with_dpp(float v) {
    return Op::of(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true)));
}
template <class Op, int L>
__device__ __forceinline__ float over_lanes(float v) {
    v = with_dpp<Op, 0xB1>(v);                        // lane ^ 1
    v = with_dpp<Op, 0x4E>(v);                        // lane ^ 2
    if constexpr (L >= 8) v = with_dpp<Op, 0x141>(v);   // lane ^ 7
    if constexpr (L >= 16) v = with_dpp<Op, 0x140>(v);  // lane ^ 15
    if constexpr (L >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = Op::of(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    if constexpr (L >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = Op::of(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    return v;
}

template <int L>
__device__ __forceinline__ int sum_over_lanes(int v) {
    return __float_as_int(over_lanes<IntSum, L>(__int_as_float(v)));
}

constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

// Maxima that pass over NaN; fmaxf quiets its operands first, an instruction more for each.
__device__ __forceinline__ float max2(float a, float b) {
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ float Max::of(float a, float b) { return max2(a, b); }
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// ---- a row
template <int L, int V, bool VEC>
__device__ __forceinline__ int expert_of(int lane, int i) {
    return VEC ? 4 * (lane + L * (i / 4)) + i % 4 : lane + L * i;
}

// The logits of the row at `row`; -infinity past the last expert, or everywhere where the row is not to be had.
template <int TYPE, int L, int V, bool VEC>
__device__ __forceinline__ void load_row(float (&l)[V], const char* row, int E, int lane, bool valid = true) {
    constexpr int SIZE = TYPE == MOE_F32 ? 4 : 2;
    row += (VEC ? 4 : 1) * lane * SIZE;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const char* at = row + L * i * SIZE;
#pragma unroll
            for (int j = 0; j < 4; ++j) l[i + j] = -INFINITY;
            if (!valid || expert_of<L, V, VEC>(lane, i) >= E) continue;
            if constexpr (TYPE == MOE_F32) {
                const v4f v = *reinterpret_cast<const v4f*>(at);
#pragma unroll
                for (int j = 0; j < 4; ++j) l[i + j] = v[j];
            } else {
                const v2i v = *reinterpret_cast<const v2i*>(at);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    l[i + j] = __uint_as_float(j & 1 ? (uint32_t)v[j / 2] & 0xFFFF0000u : (uint32_t)v[j / 2] << 16);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            l[i] = -INFINITY;
            if (valid && expert_of<L, V, VEC>(lane, i) < E) {
                const char* at = row + L * i * SIZE;
                if constexpr (TYPE == MOE_F32) l[i] = *reinterpret_cast<const float*>(at);
                else l[i] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(at) << 16);
            }
        }
    }
}

// Scores of a row as shares of their sum.  `top` is the largest logit, NaN aside; a padding row has none and shares of 0.
//   softmax: exp(l - top) as 2^(l log2 e - top log2 e), the difference rounded once: off by 2^-24 |l - top| (1 + 0.2),
//            for the rounding and for log2 e's; what the rounding of top log2 e does is the same for the whole row
//            and, below kFar, a factor of 2^(+-1/16) at most.  From 2^31 on that factor alone would pass FP32's range, so from
//            kFar on it is 2^((l - top) log2 e): off by 2^-24 |l - top| (2 + 0.2), and logits there lie 1/8 apart or are equal
//   sigmoid: 1 / (1 + 2^(-l log2 e)), which is 0 below 2^-126; where all logits are below 0, exp(l - top) / (1 + exp(l)),
//            which keeps the shares of scores that are tiny beside 1, but not beside the largest
// A NaN or, with softmax, an infinity makes the sum NaN, and the log-sum-exp NaN or infinite.  Exponentials below 2^-125 of
// the largest may be 0.
constexpr float kFar = 0x1p20f;
struct RowSum {
    float top, by, sum, inv;  // by: top log2 e, or 0; inv: 1 over the sum
    bool alive;
    __device__ __forceinline__ float lse() const {  // softmax alone
        const float v = fabsf(top) < 0x1p100f ? (by + __builtin_amdgcn_logf(sum)) * kLn2 : top;
        return alive ? v : 0.0f;
    }
};
__device__ __forceinline__ float sigmoid(float l) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * l));
}
__device__ __forceinline__ float exp_over(float l, float top) { return __builtin_amdgcn_exp2f((l - top) * kLog2e); }

// rest: of sigmoid scores, what they lack to 1 (REST alone)
template <int SCORE, int L, int V, bool REST>
__device__ __forceinline__ RowSum shares(const float (&l)[V], float (&p)[V], float (&rest)[V]) {
    RowSum r;
    float top = max2(l[0], l[1]);
#pragma unroll
    for (int i = 2; i < V; i += 2) top = max3(top, l[i], l[i + 1]);
    r.top = over_lanes<Max, L>(top);
    r.alive = r.top > -INFINITY;
    if (!r.alive) {  // padding, or NaN beside it
        bool nan = false;
#pragma unroll
        for (int i = 0; i < V; ++i) nan |= l[i] != l[i];
        r.alive = over_lanes<Max, L>(nan ? 1.0f : 0.0f) > 0.0f;
    }
    r.by = r.alive ? r.top * kLog2e : 0.0f;
    if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
        if (fabsf(r.top) < kFar || !r.alive) {
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = __builtin_amdgcn_exp2f(fmaf(l[i], kLog2e, -r.by));
        } else {
            float nan = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                p[i] = exp_over(l[i], r.top);
                nan += p[i];
            }
            nan = over_lanes<Sum, L>(nan);
            if (nan != nan && r.top < INFINITY) r.top = nan;  // for lse
        }
    } else {
        if (r.top >= 0.0f || !r.alive) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float e = __builtin_amdgcn_exp2f(-kLog2e * l[i]);
                p[i] = __builtin_amdgcn_rcpf(1.0f + e);
                if constexpr (REST) rest[i] = l[i] < -64.0f ? 1.0f : e * p[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                p[i] = exp_over(l[i], r.top);
                const float less = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[i] * kLog2e));
                p[i] *= less;
                if constexpr (REST) rest[i] = less;
            }
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += p[i];
    r.sum = over_lanes<Sum, L>(sum);
    r.inv = r.alive ? __builtin_amdgcn_rcpf(r.sum) : 0.0f;
    return r;
}

// ---- sequences
__device__ __forceinline__ int offset_at(const int64_t* off, int s, int T) {
    if (!off) return s > 0 ? T : 0;
    const int64_t o = off[s];
    return (int)(o < 0 ? 0 : o > T ? T : o);
}
// The last sequence that begins at or before `row`: -1 .. S, S where the last one ends at or before it.
__device__ __forceinline__ int sequence_of(const int64_t* off, int row, int S, int T) {
    if (!off) return 0;
    int lo = 0, hi = S + 1;  // offsets below lo are <= row, those from hi on are > row
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (offset_at(off, mid, T) <= row) lo = mid + 1;
        else hi = mid;
    }
    return lo - 1;
}

// The same of one row for a whole wave, which compares 64 offsets at a time, and the sequence's rows: in front of the first
// sequence those up to it, behind the last those from its end on.  All lanes of the wave have to be on.
struct Span {
    int s, begin, end;
};
__device__ __forceinline__ Span span_of_wave(const int64_t* off, int row, int S, int T) {
    if (!off) return {0, 0, T};
    const int lane = threadIdx.x % 64;
    int lo = 0, n = S + 1;  // the offsets in question
    Span r{-1, 0, T};
    while (n > 0) {
        const int step = (n + 63) / 64, at = lane * step;
        const int o = at < n ? offset_at(off, lo + at, T) : T;
        const int c = __popcll(__ballot(at < n && o <= row));
        if (c > 0) r.begin = __builtin_amdgcn_readlane(o, c - 1);
        if (c < 64 && c * step < n) r.end = __builtin_amdgcn_readlane(o, c);
        if (c == 0) break;
        lo += (c - 1) * step + 1;
        n = min(step - 1, n - (c - 1) * step - 1);
    }
    r.s = lo - 1;
    return r;
}
// The sequence of a row at or behind sequence s's first: often s or the next one.
__device__ __forceinline__ int sequence_from(const int64_t* off, int s, int row, int S, int T) {
    for (int i = 0; i < 3; ++i) {
        if (s >= S || row < offset_at(off, s + 1, T)) return s;
        ++s;
    }
    return sequence_of(off, row, S, T);
}

// ---- forward: sums of a tile's rows, then sums of the tiles
//
// The rows are cut into tiles, whatever the sequences.  A sequence within one tile is summed and written by a workgroup
// of its own.  What a tile has of longer ones, the tail of one that began before it and the head of one that goes on
// behind it, goes to slots, and a second kernel adds a sequence's parts in the order of their tiles.  So a workgroup has
// two parts to sum at most, however many sequences there are, and nothing depends on the order of workgroups or of
// atomics (those on counts are whole numbers).
// Bound by memory where rows are many (65536 x 384 FP32: 22.5 us, 4.6 TB/s, and 6 to join) and by the chain of a
// workgroup where they are few (128 x 256: 6.0 us): loads, two instructions an exponential, sums over lanes and waves.
// Two rows of a group are loaded together; more in flight gained nothing.
// The part of sequence s in tile b has slot b + s (from one part to the next b or s grows, so no two share one) or, with
// more sequences than tiles, 2 b and, where the sequence begins in the tile, 2 b + 1.
__device__ __forceinline__ int64_t slot_of(int b, int s, bool head, bool many) {
    return many ? 2 * (int64_t)b + head : (int64_t)b + s;
}
struct Slot {  // floats and ints of one part: shares [E], counts [E], then rows and z
    static __host__ __device__ __forceinline__ int64_t words(int E) { return 2 * (int64_t)E + 2; }
};

// Waves of a workgroup of the first kernel; their sums, one per expert, stand side by side in LDS.
template <int V>
constexpr int kWaves = V > 8 ? 8 : 16;

constexpr int kShortWaves = 4;

template <int W>
struct RowSums {  // in LDS
    int E;
    float* share;  // [W][E]
    int* count;    // [E]
    int* rows;     // [W]
    float* z;      // [W]
    __device__ __forceinline__ RowSums(float* smem, int E)
        : E(E), share(smem), count(reinterpret_cast<int*>(smem + W * E)), rows(count + E), z(reinterpret_cast<float*>(rows + W)) {}
    static size_t bytes(int E) { return ((size_t)(W + 1) * E + 2 * W) * 4; }
    __device__ __forceinline__ float share_of(int e) const {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += share[w * E + e];
        return v;
    }
    __device__ __forceinline__ void row_totals(int& n, float& zz) const {
        n = 0;
        zz = 0.0f;
        for (int w = 0; w < W; ++w) n += rows[w], zz += z[w];
    }
};

// Sums of rows [row, end), of the whole workgroup; the caller's next barrier is behind the last read of them.
template <int TYPE, int SCORE, int L, int V, bool VEC, int W>
__device__ __forceinline__ void sum_rows(const BalanceArgs& a, int row, int end, const RowSums<W>& out) {
    constexpr int THREADS = W * 64, GROUPS = THREADS / L;
    constexpr int U = V > 8 ? 1 : 2;  // rows of a group that are loaded together
    const int tid = threadIdx.x, lane = tid % L, group = tid / L, wave = tid / 64;
    for (int e = tid; e < a.E; e += THREADS) out.count[e] = 0;
    const int64_t id0 = (int64_t)row * a.k, ids = (int64_t)(end - row) * a.k;
    const int64_t first_id = tid < ids ? a.topk_idx[id0 + tid] : -1;
    float acc[V], z = 0.0f;
    int rows = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    if (a.logits) {
        const char* base = static_cast<const char*>(a.logits);
        const int64_t pitch = a.stride * (TYPE == MOE_F32 ? 4 : 2);
        for (int t = row + group; t < end; t += U * GROUPS) {
            float l[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u)
                load_row<TYPE, L, V, VEC>(l[u], base + (int64_t)(t + u * GROUPS) * pitch, a.E, lane, t + u * GROUPS < end);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float p[V];
                const RowSum r = shares<SCORE, L, V, false>(l[u], p, p);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = fmaf(p[i], r.inv, acc[i]);
                rows += r.alive;
                if (SCORE == MOE_SCORE_SOFTMAX && a.z) {
                    const float lse = r.lse();
                    z = fmaf(lse, lse, z);
                }
            }
        }
    }
    // the groups of a wave, then the waves
    if constexpr (L < 64) {
#pragma unroll
        for (int d = L; d < 64; d *= 2) {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += __shfl_xor(acc[i], d);
            rows += __shfl_xor(rows, d);
            z += __shfl_xor(z, d);
        }
    }
    if (tid % 64 < L) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = expert_of<L, V, VEC>(lane, i);
            if (e < a.E) out.share[wave * a.E + e] = acc[i];
        }
        if (lane == 0) {
            out.rows[wave] = rows;
            out.z[wave] = z;
        }
    }
    __syncthreads();
    if (first_id >= 0 && first_id < a.E) atomicAdd(&out.count[first_id], 1);
    for (int64_t i = tid + THREADS; i < ids; i += THREADS) {
        const int64_t e = a.topk_idx[id0 + i];
        if (e >= 0 && e < a.E) atomicAdd(&out.count[e], 1);
    }
    __syncthreads();
}

template <int TYPE, int SCORE, int L, int V, bool VEC, int W>
__global__ __launch_bounds__(W * 64) void balance_rows_kernel(BalanceArgs a, int tile, int tiles, float* parts,
                                                                      uint32_t* tickets) {
    extern __shared__ float smem[];
    __shared__ float cross_part[W];
    __shared__ int count_part[W];
    constexpr int THREADS = W * 64;
    const RowSums<W> sums(smem, a.E);
    const int tid = threadIdx.x;
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (block < tiles) {  // none where all rows are of one tile
        const int b = (int)block, row = b * tile, last = min(row + tile, a.T);
        if (tid == 0 && tickets && b < a.S) tickets[b] = 0;
        Span span = span_of_wave(a.seq_offsets, row, a.S, a.T);
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
            int from = row, to = min(span.end, last);
            bool has = span.begin < row;
            if (part == 1) {
                if (last == a.T) break;
                if (span.end <= last) span = span_of_wave(a.seq_offsets, last - 1, a.S, a.T);
                from = span.begin;
                to = last;
                has = span.begin >= row && span.end > last;
            }
            if (!has || span.s < 0 || span.s >= a.S) continue;
            sum_rows<TYPE, SCORE, L, V, VEC, W>(a, from, to, sums);
            float* out = parts + slot_of(b, span.s, part == 1, a.S > tiles) * Slot::words(a.E);
            for (int e = tid; e < a.E; e += THREADS) {
                out[e] = sums.share_of(e);
                reinterpret_cast<int*>(out)[a.E + e] = sums.count[e];
            }
            if (tid == 0) {
                int n;
                float z;
                sums.row_totals(n, z);
                reinterpret_cast<int*>(out)[2 * a.E] = n;
                out[2 * a.E + 1] = z;
            }
            __syncthreads();
        }
        return;
    }
    const int64_t s = block - tiles;
    if (s >= a.S) return;
    const int from = offset_at(a.seq_offsets, (int)s, a.T), to = max(from, offset_at(a.seq_offsets, (int)s + 1, a.T));
    if (tiles > 0 && to > from && from / tile != (to - 1) / tile) return;  // the tiles'
    sum_rows<TYPE, SCORE, L, V, VEC, W>(a, from, to, sums);
    int n;
    float z;
    sums.row_totals(n, z);
    float cross = 0.0f;
    int total = 0;
    for (int e = tid; e < a.E; e += THREADS) {
        const int count = sums.count[e];
        const float share = n > 0 ? sums.share_of(e) / (float)n : 0.0f;
        if (a.counts) a.counts[s * a.E + e] = count;
        if (a.share) a.share[s * a.E + e] = share;
        if (count > 0) cross += (float)count * share;
        total += count;
    }
    if (tid == 0) {
        if (a.rows) a.rows[s] = n;
        if (a.z) a.z[s] = n > 0 ? z / (float)n : 0.0f;
    }
    if (!a.loss) return;
    cross = over_lanes<Sum, 64>(cross);
    total = sum_over_lanes<64>(total);
    if (tid % 64 == 0) {
        cross_part[tid / 64] = cross;
        count_part[tid / 64] = total;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < W; ++w) cross += cross_part[w], total += count_part[w];
        a.loss[s] = total > 0 ? (float)a.E * cross / (float)total : 0.0f;
    }
}

// The sequence that a workgroup of the second kernel joins, s < 0 for none: the `index`th or, where there are more
// sequences than tiles, the one that crosses its first border of two tiles there; its tiles are [first, end).
struct Longer {
    int s, first, end;
};
__device__ __forceinline__ Longer longer_of(const BalanceArgs& a, int64_t index, int tile, int borders) {
    const Longer none{-1, 0, 0};
    int s = (int)index, from, to;
    if (borders == 0) {
        if (index >= a.S) return none;
        from = offset_at(a.seq_offsets, s, a.T);
        to = offset_at(a.seq_offsets, s + 1, a.T);
    } else {
        if (index >= borders) return none;
        const int border = (s + 1) * tile;
        const Span span = span_of_wave(a.seq_offsets, border, a.S, a.T);
        s = span.s;
        from = span.begin;
        to = span.end;
        if (s < 0 || s >= a.S || from >= border || from / tile != border / tile - 1) return none;
    }
    const int first = from / tile, end = (to - 1) / tile + 1;
    if (to <= from || end == first + 1) return none;  // written already
    return {s, first, end};
}

// One workgroup per sequence and kColumns experts; the last of a sequence to arrive adds up the loss.
constexpr int kColumns = 16, kJoinThreads = 1024;
static_assert(kMaxGateExperts / kColumns <= 64, "a lane for each of a sequence's workgroups");
static_assert(kMaxGateExperts <= kJoinThreads, "a lane for each expert");
__global__ __launch_bounds__(kJoinThreads) void balance_long_join_kernel(BalanceArgs a, int tile, const float* parts,
                                                                         uint32_t* tickets, float* sums) {
    __shared__ float share_part[kJoinThreads / kColumns][kColumns], z_part[kJoinThreads / kColumns];
    __shared__ int count_part[kJoinThreads / kColumns][kColumns], rows_part[kJoinThreads / kColumns];
    constexpr int LANES = kJoinThreads / kColumns;
    const int chunks = (a.E + kColumns - 1) / kColumns;
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int chunk = (int)(block % chunks);
    const Longer q = longer_of(a, block / chunks, tile, 0);
    if (q.s < 0) return;
    const int s = q.s, first = q.first, end = q.end;
    const int col = threadIdx.x % kColumns, part = threadIdx.x / kColumns, e = chunk * kColumns + col;
    const int64_t words = Slot::words(a.E);
    float share = 0.0f, z = 0.0f;
    int count = 0, rows = 0;
    const int at = min(e, a.E - 1);
#pragma unroll 8
    for (int b = first + part; b < end; b += LANES) {
        const float* in = parts + slot_of(b, s, b == first, false) * words;
        share += in[at];
        count += reinterpret_cast<const int*>(in)[a.E + at];
        if (col == 0) {
            rows += reinterpret_cast<const int*>(in)[2 * a.E];
            z += in[2 * a.E + 1];
        }
    }
    share_part[part][col] = share;
    count_part[part][col] = count;
    if (col == 0) {
        rows_part[part] = rows;
        z_part[part] = z;
    }
    __syncthreads();
    if (threadIdx.x >= 64) return;
    // one wave, whose lanes of a column take its parts in turn
    rows = (int)threadIdx.x < LANES ? rows_part[threadIdx.x] : 0;
    z = (int)threadIdx.x < LANES ? z_part[threadIdx.x] : 0.0f;
    rows = sum_over_lanes<64>(rows);
    z = over_lanes<Sum, 64>(z);
    share = 0.0f;
    count = 0;
#pragma unroll 4
    for (int q = part; q < LANES; q += 64 / kColumns) {
        share += share_part[q][col];
        count += count_part[q][col];
    }
#pragma unroll
    for (int d = kColumns; d < 64; d *= 2) {
        share += __shfl_xor(share, d);
        count += __shfl_xor(count, d);
    }
    share = rows > 0 ? share / (float)rows : 0.0f;
    const bool mine = threadIdx.x < kColumns && e < a.E;
    if (mine) {
        if (a.counts) a.counts[(int64_t)s * a.E + e] = count;
        if (a.share) a.share[(int64_t)s * a.E + e] = share;
    }
    if (chunk == 0 && threadIdx.x == 0) {
        if (a.rows) a.rows[s] = rows;
        if (a.z) a.z[s] = rows > 0 ? z / (float)rows : 0.0f;
    }
    if (!a.loss) return;
    const float cross = over_lanes<Sum, 64>(mine && count > 0 ? (float)count * share : 0.0f);
    const int total = sum_over_lanes<64>(mine ? count : 0);
    float* out = sums + ((int64_t)s * chunks + chunk) * 2;
    uint32_t before = 0;
    if (threadIdx.x == 0) {
        __hip_atomic_store(out, cross, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(out + 1, __int_as_float(total), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        before = __hip_atomic_fetch_add(&tickets[s], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane(before) != (uint32_t)chunks - 1) return;
    const float* all = sums + ((int64_t)s * chunks + min((int)threadIdx.x, chunks - 1)) * 2;
    const float part_cross = __hip_atomic_load(all, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const int part_total = __float_as_int(__hip_atomic_load(all + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    const bool has = (int)threadIdx.x < chunks;
    const float v = over_lanes<Sum, 64>(has ? part_cross : 0.0f);
    const int n = sum_over_lanes<64>(has ? part_total : 0);
    if (threadIdx.x == 0) a.loss[s] = n > 0 ? (float)a.E * v / (float)n : 0.0f;
}

// One workgroup per sequence, or per border where there are more sequences than tiles: a lane for every expert and, of few
// experts, several lanes for its parts in turn.
__global__ __launch_bounds__(kJoinThreads) void balance_short_join_kernel(BalanceArgs a, int tile, int borders,
                                                                          const float* parts) {
    __shared__ float share_part[kJoinThreads], cross_part[kJoinThreads / 64];
    __shared__ int count_part[kJoinThreads], total_part[kJoinThreads / 64];
    const Longer q = longer_of(a, (int64_t)blockIdx.y * gridDim.x + blockIdx.x, tile, borders);
    if (q.s < 0) return;
    const int width = (a.E + 63) / 64 * 64, lanes = blockDim.x / width;
    const int e = threadIdx.x % width, part = threadIdx.x / width;
    const int64_t words = Slot::words(a.E);
    const int at = min(e, a.E - 1);
    float share = 0.0f, z = 0.0f;
    int count = 0, rows = 0;
#pragma unroll 8
    for (int b = q.first + part; b < q.end; b += lanes) {
        const float* in = parts + slot_of(b, q.s, b == q.first, borders > 0) * words;
        share += in[at];
        count += reinterpret_cast<const int*>(in)[a.E + at];
    }
    for (int b = q.first + (int)threadIdx.x % 64; b < q.end; b += 64) {  // each wave for itself
        const float* in = parts + slot_of(b, q.s, b == q.first, borders > 0) * words;
        rows += reinterpret_cast<const int*>(in)[2 * a.E];
        z += in[2 * a.E + 1];
    }
    rows = sum_over_lanes<64>(rows);
    z = over_lanes<Sum, 64>(z);
    share_part[threadIdx.x] = share;
    count_part[threadIdx.x] = count;
    __syncthreads();
    float cross = 0.0f;
    int total = 0;
    if (part == 0 && e < a.E) {
        for (int l = 1; l < lanes; ++l) {
            share += share_part[l * width + e];
            count += count_part[l * width + e];
        }
        share = rows > 0 ? share / (float)rows : 0.0f;
        if (a.counts) a.counts[(int64_t)q.s * a.E + e] = count;
        if (a.share) a.share[(int64_t)q.s * a.E + e] = share;
        if (count > 0) cross = (float)count * share;
        total = count;
    }
    if (threadIdx.x == 0) {
        if (a.rows) a.rows[q.s] = rows;
        if (a.z) a.z[q.s] = rows > 0 ? z / (float)rows : 0.0f;
    }
    if (!a.loss) return;
    cross = over_lanes<Sum, 64>(cross);
    total = sum_over_lanes<64>(total);
    if (threadIdx.x % 64 == 0) {
        cross_part[threadIdx.x / 64] = cross;
        total_part[threadIdx.x / 64] = total;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < width / 64; ++w) cross += cross_part[w], total += total_part[w];
        a.loss[q.s] = total > 0 ? (float)a.E * cross / (float)total : 0.0f;
    }
}

// Rows of a tile.  One tile, and one launch, where sequences have some 192 rows and all together 1024 at most (us for one
// tile / several, E = 256: 300 rows in 5 sequences 4.9 / 10.0, 1000 in 7 7.4 / 10.7; in one sequence 190 rows 7.9 / 8.0,
// 256 9.5 / 8.6, 1000 26 / 8.8).  Else a tile for every compute unit, and no more parts than the second kernel adds quickly
// (65536 x 384: 28.4 us for tiles of 256 rows, 41.8 for 512, 27.9 for 128; 16384 x 256: 12.1, 11.7, 16.8 for 64, 128, 32).
// Measured at 256 and 384 experts, and taken for any number.
int tile_rows(int T, int S) {
    int tile = 16;
    if (T <= 1024 && T <= 192 * (int64_t)S) return 1024;
    while (tile < 1024 && (int64_t)tile * 256 < T) tile *= 2;
    return tile;
}

// Sequences of so many tiles or more, if all are as long, are joined by 16 experts a workgroup, shorter ones by one each:
// a workgroup that takes a ticket costs the others' time (its release writes back the cache), so that 13 sequences of 20
// tiles take 14.7 us to 17.4, 50 of 5 13.4 to 27.4; one of 256, which leaves a single workgroup, is the other way about.
constexpr int kLong = 64;
struct BalanceLayout {
    int tile, tiles;
    bool long_join;
    size_t parts = 0, tickets = 0, sums = 0, total = 0;
};
BalanceLayout balance_layout(int T, int E, int S) {
    BalanceLayout l;
    l.tile = tile_rows(T, S);
    l.tiles = (int)(((int64_t)T + l.tile - 1) / l.tile);
    size_t o = 0;
    auto take = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes, kAlign); return at; };
    l.long_join = l.tiles >= kLong * (int64_t)S;
    l.parts = take(((size_t)l.tiles + std::max(1, std::min(l.tiles, S))) * Slot::words(E) * 4);
    l.tickets = take((size_t)(l.long_join ? S : 0) * 4);
    l.sums = take((size_t)(l.long_join ? S : 0) * ((E + kColumns - 1) / kColumns) * 8);
    l.total = o;
    return l;
}

// ---- backward
//
// With g[e] = d_loss E counts[e] / (sum of counts) / rows, and q its mean under p:
//   softmax  p (g - q),  sigmoid  p (1 - s) (g - q)
// What all experts have in common falls out of g - q, so g is formed from E counts[e] - sum of counts, in whole numbers:
// the gradient of an even load is then 0 and that of a nearly even one keeps its bits.
// z adds p * 2 lse d_z / rows.  The weights w = scale * r, r = s over the sum of the chosen (or s), add at the chosen
//   renormalised:  softmax  scale r (d - m),  sigmoid  scale r (1 - s) (d - m),  m = sum of r d
//   else:          softmax  scale p d, and -p * (sum of scale p d) at every expert;  sigmoid  scale s (1 - s) d
//
// A row is read and written once; what its sequence needs stays in registers while a group's rows are of it.  65536 x 384
// FP32 takes 48 us (207 MB, 4.3 TB/s), 16384 x 256 BF16 in 13 sequences 12.0, bound by vector instructions.  Scores of the
// chosen are gathered and their gradients scattered in LDS, not by comparing every id with every expert (with that and
// exponentials of more instructions 75).
template <int TYPE, int SCORE, int L, int V, bool VEC, int KV>
__global__ __launch_bounds__(kThreads) void gate_grad_kernel(GateGradArgs a, int rows_per_group) {
    constexpr int GROUPS = kThreads / L, SIZE = TYPE == MOE_F32 ? 4 : 2;
    // What a group's row adds at the experts it chose, by expert (zeros between rows), and the row's scores (softmax) or
    // logits for its chosen experts to be read from.  A group's lanes are of one wave, whose LDS instructions are done in
    // their order (wave_exchange has the compiler keep it), and an instruction's additions to one place in the lanes' order.
    __shared__ __attribute__((aligned(16))) float sums_of_rows[GROUPS][L * V], row_of_group[GROUPS][L * V];
    const int lane = threadIdx.x % L, group = threadIdx.x / L;
    float* own = sums_of_rows[group];
    float* values = row_of_group[group];
#pragma unroll
    for (int i = 0; i < V; ++i) own[lane + L * i] = 0.0f;
    wave_exchange();
    const int64_t first = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * GROUPS * rows_per_group;
    if (first >= a.T) return;
    int64_t t = first + group;
    const char* in = static_cast<const char*>(a.logits) + t * a.stride * SIZE;
    char* out = static_cast<char*>(a.d_logits) + t * a.E * SIZE;
    int64_t at_k = t * a.k + lane;
    // the sequence of the last row, here of the wave's first one, and its rows; `known`: what of it the rows need is loaded.
    // Looked up in front of the loop, where lanes of groups without a row are on too: the search has all 64 take part.
    const Span span = span_of_wave(a.seq_offsets, (int)min(first + threadIdx.x / 64 * (64 / L), (int64_t)a.T), a.S, a.T);
    int s = span.s, begin = span.begin, end = span.end;
    bool known = false;
    float pull[V], zpull = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) pull[i] = 0.0f;
    for (int step = 0; step < rows_per_group && t < a.T; ++step, t += GROUPS, in += GROUPS * a.stride * SIZE,
             out += (int64_t)GROUPS * a.E * SIZE, at_k += GROUPS * a.k) {
        float l[V], p[V], dw[KV];
        int id[KV];
        load_row<TYPE, L, V, VEC>(l, in, a.E, lane);
        if (a.d_topk_w) {
#pragma unroll
            for (int q = 0; q < KV; ++q) id[q] = -1, dw[q] = 0.0f;
#pragma unroll
            for (int q = 0; q < KV; ++q) {
                if (q > 0 && q * L >= a.k) break;
                if (lane + q * L < a.k) {
                    const int64_t e = a.topk_idx[at_k + q * L];
                    id[q] = (uint64_t)e < (uint64_t)a.E ? (int)e : -1;
                    dw[q] = a.scale * a.d_topk_w[at_k + q * L];
                }
            }
        }
        if (t < begin || t >= end) {
            known = false;
            s = sequence_from(a.seq_offsets, max(s, 0), (int)t, a.S, a.T);
            begin = offset_at(a.seq_offsets, min(s, a.S), a.T);
            if (s == 0 && t < begin) {  // in front of the first sequence
                s = -1;
                end = begin;
                begin = 0;
            } else {
                end = s < a.S ? offset_at(a.seq_offsets, s + 1, a.T) : a.T;
            }
        }
        if (s < 0 || s >= a.S) continue;
        if (!known) {
            known = true;
            const float n = a.rows ? (float)a.rows[s] : 0.0f;
            if (a.d_loss) {
                int c[V], low = 0, high = 0;  // halves of the sum, which may pass 32 bits
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = expert_of<L, V, VEC>(lane, i);
                    c[i] = e < a.E ? a.counts[(int64_t)s * a.E + e] : 0;
                    low += c[i] & 0xFFFF;
                    high += c[i] >> 16;
                }
                const double total = 65536.0 * sum_over_lanes<L>(high) + sum_over_lanes<L>(low);
                const float by = n > 0.0f && total != 0.0 ? a.d_loss[s] / n / (float)total : 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) pull[i] = by * (float)fma((double)c[i], (double)a.E, -total);  // exact before it is rounded
            }
            zpull = a.d_z && n > 0.0f ? 2.0f * a.d_z[s] / n : 0.0f;
        }

        float less[V];  // of sigmoid scores
        const RowSum r = shares<SCORE, L, V, SCORE == MOE_SCORE_SIGMOID>(l, p, less);
        float common = 0.0f;  // what falls on every expert by its share
        if (a.d_loss) {
#pragma unroll
            for (int i = 0; i < V; ++i) common = fmaf(p[i], pull[i], common);
            common = -over_lanes<Sum, L>(common) * r.inv;
        }
        if (SCORE == MOE_SCORE_SOFTMAX && a.d_z) common = fmaf(zpull, r.lse(), common);
        if (a.d_topk_w) {
#pragma unroll
            for (int i = 0; i < V; ++i) values[expert_of<L, V, VEC>(lane, i)] = SCORE == MOE_SCORE_SOFTMAX ? p[i] : l[i];
            wave_exchange();
            // the chosen's scores and, of sigmoid ones, what they lack to 1; where there is no score, as of an id that is none or
            // a masked logit's, d_topk_w may be anything
            float w[KV], rest[KV];
            float sum = 0.0f, m = 0.0f;
#pragma unroll
            for (int q = 0; q < KV; ++q) w[q] = 0.0f, rest[q] = 1.0f;
#pragma unroll
            for (int q = 0; q < KV; ++q) {
                if (q > 0 && q * L >= a.k) break;
                if (id[q] >= 0) {
                    const float v = values[id[q]];
                    if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
                        w[q] = v;
                    } else {
                        w[q] = sigmoid(v);
                        rest[q] = sigmoid(-v);
                    }
                }
                sum += w[q];
                if (w[q] != 0.0f) m = fmaf(w[q], dw[q], m);
            }
            sum = over_lanes<Sum, L>(sum);
            m = over_lanes<Sum, L>(m);
            if (a.renorm) {
                // far below the row's largest, or sigmoid scores of which smaller ones may be lost: formed over the largest of them
                if (sum < (SCORE == MOE_SCORE_SOFTMAX ? 0x1p-80f : 0.5f)) {
                    float top = -INFINITY, lk[KV];
                    wave_exchange();
#pragma unroll
                    for (int i = 0; i < V; ++i) values[expert_of<L, V, VEC>(lane, i)] = l[i];
                    wave_exchange();
#pragma unroll
                    for (int q = 0; q < KV; ++q) {
                        lk[q] = id[q] >= 0 ? values[id[q]] : -INFINITY;
                        top = max2(top, lk[q]);
                    }
                    top = over_lanes<Max, L>(top);
                    sum = m = 0.0f;
#pragma unroll
                    for (int q = 0; q < KV; ++q) {
                        w[q] = lk[q] > -INFINITY ? exp_over(lk[q], top) : 0.0f;
                        if constexpr (SCORE == MOE_SCORE_SIGMOID) w[q] *= rest[q];  // 1 / (1 + exp(l))
                        sum += w[q];
                        if (w[q] != 0.0f) m = fmaf(w[q], dw[q], m);
                    }
                    sum = over_lanes<Sum, L>(sum);
                    m = over_lanes<Sum, L>(m);
                }
                const float inv = sum != 0.0f ? __builtin_amdgcn_rcpf(sum) : 0.0f;
                m *= inv;
#pragma unroll
                for (int q = 0; q < KV; ++q) w[q] *= inv;
            } else {
                if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
                    common = fmaf(-m, r.inv, common);
#pragma unroll
                    for (int q = 0; q < KV; ++q) w[q] *= r.inv;
                }
                m = 0.0f;
            }
#pragma unroll
            for (int q = 0; q < KV; ++q) {
                if (q > 0 && q * L >= a.k) break;
                if (id[q] >= 0 && w[q] != 0.0f) atomicAdd(&own[id[q]], w[q] * (dw[q] - m) * rest[q]);
            }
        }
        float g[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            g[i] = p[i] * fmaf(pull[i], r.inv, common * r.inv);
            if constexpr (SCORE == MOE_SCORE_SIGMOID) g[i] *= less[i];
        }
        if (a.d_topk_w) {
            wave_exchange();
#pragma unroll
            for (int i = 0; i < V; ++i) g[i] += own[expert_of<L, V, VEC>(lane, i)];
            wave_exchange();
#pragma unroll
            for (int q = 0; q < KV; ++q) {
                if (q > 0 && q * L >= a.k) break;
                if (id[q] >= 0) own[id[q]] = 0.0f;
            }
        }
        if (!(fabsf(common * r.inv) < INFINITY)) {  // a masked expert has a gradient of 0 beside a NaN too
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (l[i] == -INFINITY) g[i] = 0.0f;
        }
        char* at = out + (VEC ? 4 : 1) * lane * SIZE;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                if (expert_of<L, V, VEC>(lane, i) >= a.E) continue;
                if constexpr (TYPE == MOE_F32)
                    *reinterpret_cast<v4f*>(at + L * i * SIZE) = v4f{g[i], g[i + 1], g[i + 2], g[i + 3]};
                else
                    *reinterpret_cast<v2i*>(at + L * i * SIZE) =
                        v2i{(int)pack_bf16(g[i], g[i + 1]), (int)pack_bf16(g[i + 2], g[i + 3])};
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (expert_of<L, V, VEC>(lane, i) >= a.E) continue;
                if constexpr (TYPE == MOE_F32) *reinterpret_cast<float*>(at + L * i * SIZE) = g[i];
                else *reinterpret_cast<uint16_t*>(at + L * i * SIZE) = (uint16_t)pack_bf16(g[i], g[i]);
            }
        }
    }
}

// ---- choice of the lanes of a row
bool vector_rows(const void* base, int64_t stride, int E, int type) {
    const uintptr_t size = type == MOE_F32 ? 16 : 8;
    return E % 4 == 0 && stride % 4 == 0 && reinterpret_cast<uintptr_t>(base) % size == 0;
}

template <int TYPE, int SCORE, int L, int V, bool VEC>
void parts_go(const BalanceArgs& a, const BalanceLayout& l, char* ws, hipStream_t stream) {
    // Four waves for short sequences, of which most of a larger workgroup would have no rows (16384 rows in 4000 18 us to
    // 53), longer ones where there are many (300 of 55 rows 14.0 to 18.9; but 5 of 60 5.9 to 4.9).
    const int tiles = l.tiles > 1 ? l.tiles : 0;
    auto launch = [&](auto waves) {
        constexpr int W = decltype(waves)::value;
        hipLaunchKernelGGL((balance_rows_kernel<TYPE, SCORE, L, V, VEC, W>), wide_grid((int64_t)tiles + a.S), dim3(W * 64),
                           RowSums<W>::bytes(a.E), stream, a, l.tile, tiles, reinterpret_cast<float*>(ws + l.parts),
                           l.long_join ? reinterpret_cast<uint32_t*>(ws + l.tickets) : nullptr);
    };
    if (a.S > 1 && a.T / a.S <= (a.S >= 64 ? 64 : 32)) launch(std::integral_constant<int, kShortWaves>{});
    else launch(std::integral_constant<int, kWaves<V>>{});
}
template <int TYPE, int SCORE, int L, int V, bool VEC, int KV>
void grad_go(const GateGradArgs& a, hipStream_t stream) {
    // rows side by side while there are workgroups to have, then several to a group, which load a sequence's counts once
    int per = 1;
    while (per < 8 && (int64_t)kThreads / L * per * 1024 < a.T) per *= 2;
    const int rows = kThreads / L * per;
    hipLaunchKernelGGL((gate_grad_kernel<TYPE, SCORE, L, V, VEC, KV>), wide_grid(((int64_t)a.T + rows - 1) / rows),
                       dim3(kThreads), 0, stream, a, per);
}

// f(type, score, lanes, values, vector loads, chosen ids per lane) as compile-time constants
template <int N>
using Int = std::integral_constant<int, N>;
template <class F>
void with_lanes(int E, F f) {
    if (E <= 32) f(Int<8>{}, Int<4>{}, Int<4>{});
    else if (E <= 64) f(Int<8>{}, Int<8>{}, Int<8>{});
    else if (E <= 128) f(Int<16>{}, Int<8>{}, Int<4>{});
    else if (E <= 256) f(Int<32>{}, Int<8>{}, Int<2>{});
    else if (E <= 384) f(Int<32>{}, Int<12>{}, Int<2>{});
    else if (E <= 512) f(Int<64>{}, Int<8>{}, Int<1>{});
    else f(Int<64>{}, Int<16>{}, Int<1>{});
}
template <class F>
void with_row(int type, int score, bool vec, int E, F f) {
    auto lanes = [&](auto t, auto s, auto v) { with_lanes(E, [&](auto l, auto n, auto kv) { f(t, s, v, l, n, kv); }); };
    auto vecs = [&](auto t, auto s) {
        if (vec) lanes(t, s, Int<1>{});
        else lanes(t, s, Int<0>{});
    };
    auto scores = [&](auto t) {
        if (score == MOE_SCORE_SOFTMAX) vecs(t, Int<MOE_SCORE_SOFTMAX>{});
        else vecs(t, Int<MOE_SCORE_SIGMOID>{});
    };
    if (type == MOE_F32) scores(Int<MOE_F32>{});
    else scores(Int<MOE_BF16>{});
}

}  // namespace

size_t balance_workspace(int T, int E, int S) { return balance_layout(T, E, S).total; }

hipError_t launch_balance(const BalanceArgs& a, void* ws, hipStream_t stream) {
    const BalanceLayout l = balance_layout(a.T, a.E, a.S);
    char* base = static_cast<char*>(ws);
    with_row(a.logits_type, a.score, vector_rows(a.logits, a.stride, a.E, a.logits_type), a.E,
             [&](auto t, auto s, auto v, auto lanes, auto n, auto) {
                 parts_go<decltype(t)::value, decltype(s)::value, decltype(lanes)::value, decltype(n)::value,
                          (bool)decltype(v)::value>(a, l, base, stream);
             });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (l.tiles <= 1) return hipSuccess;
    const float* parts = reinterpret_cast<const float*>(base + l.parts);
    if (l.long_join) {
        const int64_t chunks = (a.E + kColumns - 1) / kColumns;
        hipLaunchKernelGGL(balance_long_join_kernel, wide_grid(chunks * a.S), dim3(kJoinThreads), 0, stream, a, l.tile, parts,
                           reinterpret_cast<uint32_t*>(base + l.tickets), reinterpret_cast<float*>(base + l.sums));
    } else {
        const int borders = a.S > l.tiles ? l.tiles - 1 : 0;
        const int width = (a.E + 63) / 64 * 64, lanes = kJoinThreads / width;
        // no more lanes for an expert than its sequence has parts, if all are as long
        const int threads = width * std::max(1, std::min(lanes, l.tiles / a.S));
        hipLaunchKernelGGL(balance_short_join_kernel, wide_grid(borders ? borders : a.S), dim3((unsigned)threads), 0, stream,
                           a, l.tile, borders, parts);
    }
    return hipGetLastError();
}

hipError_t launch_gate_grad(const GateGradArgs& a, hipStream_t stream) {
    const bool vec = vector_rows(a.logits, a.stride, a.E, a.logits_type) && vector_rows(a.d_logits, a.E, a.E, a.logits_type);
    with_row(a.logits_type, a.score, vec, a.E, [&](auto t, auto s, auto v, auto lanes, auto n, auto kv) {
        grad_go<decltype(t)::value, decltype(s)::value, decltype(lanes)::value, decltype(n)::value,
                (bool)decltype(v)::value, decltype(kv)::value>(a, stream);
    });
    return hipGetLastError();
}

}  // namespace moe
