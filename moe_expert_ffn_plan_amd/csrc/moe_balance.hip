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
constexpr int kWaves = kThreads / 64;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// ---- reductions over each L neighbouring lanes, the result in all of them
struct Sum {
    static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
struct Max {
    static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); }
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

// ---- a row
template <int TYPE>
__device__ __forceinline__ float load1(const void* base, int64_t i) {
    if constexpr (TYPE == MOE_F32) return static_cast<const float*>(base)[i];
    else return __uint_as_float((uint32_t)static_cast<const uint16_t*>(base)[i] << 16);
}

template <int L, int V, bool VEC>
__device__ __forceinline__ int expert_of(int lane, int i) {
    return VEC ? 4 * (lane + L * (i / 4)) + i % 4 : lane + L * i;
}

// The logits of one row; -infinity past the last expert.
template <int TYPE, int L, int V, bool VEC>
__device__ __forceinline__ void load_row(float (&l)[V], const void* base, int64_t at, int E, int lane) {
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const int e = 4 * (lane + L * (i / 4));
            const int64_t from = at + (e < E ? e : 0);
            if constexpr (TYPE == MOE_F32) {
                const v4f v = *reinterpret_cast<const v4f*>(static_cast<const float*>(base) + from);
#pragma unroll
                for (int j = 0; j < 4; ++j) l[i + j] = v[j];
            } else {
                const v2i v = *reinterpret_cast<const v2i*>(static_cast<const uint16_t*>(base) + from);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    l[i + j] = __uint_as_float(j & 1 ? (uint32_t)v[j / 2] & 0xFFFF0000u : (uint32_t)v[j / 2] << 16);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) l[i] = load1<TYPE>(base, at + min(lane + L * i, E - 1));
    }
}
template <int L, int V, bool VEC>
__device__ __forceinline__ void mask_row(float (&l)[V], int E, int lane) {
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (expert_of<L, V, VEC>(lane, i) >= E) l[i] = -INFINITY;
}

// Scores of a row as shares of their sum.  `top` is the largest logit, +infinity where there is a NaN and -infinity
// in a padding row, whose shares are 0.  lse: the logarithm of the sum of exponentials (softmax).
//   softmax: e = exp(l - top)
//   sigmoid: with a = exp(-|l|), 1 / (1 + a) or a / (1 + a); where all logits are negative both sides of the division
//            are formed over exp(top), so that shares of tiny scores keep their bits
struct RowSum {
    float top, lse, inv;  // inv: 1 over the sum, formed over exp(top)
    bool alive;
};
template <int SCORE, int L, int V>
__device__ __forceinline__ RowSum shares(const float (&l)[V], float (&p)[V]) {
    RowSum r;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, l[i] == l[i] ? l[i] : INFINITY);
    r.top = over_lanes<Max, L>(top);
    r.alive = r.top > -INFINITY;
    float sum = 0.0f;
    if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
        const float by = r.alive ? r.top : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = expf(l[i] - by);
            sum += p[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float a = expf(-fabsf(l[i]));
            p[i] = (l[i] >= 0.0f ? 1.0f : a) / (1.0f + a);
        }
        if (r.top < 0.0f && r.alive) {
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = expf(l[i] - r.top) / (1.0f + expf(l[i]));
        }
#pragma unroll
        for (int i = 0; i < V; ++i) sum += p[i];
    }
    sum = over_lanes<Sum, L>(sum);
    r.lse = SCORE == MOE_SCORE_SOFTMAX && r.alive ? r.top + logf(sum) : 0.0f;
    r.inv = r.alive ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] *= r.inv;
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

// ---- forward: sums of a tile's rows, then sums of the tiles
//
// Tiles of `tile` rows, whatever the sequences.  The part of sequence s in tile b goes to slot b + s: from one part to
// the next b or s grows, so no two parts share a slot, and there are at most tiles + S of them.  The second kernel adds
// a sequence's parts in the order of their tiles; nothing depends on the order of workgroups or of atomics (those on
// counts are whole numbers).
struct Slot {  // floats and ints of one part: shares [E], counts [E], then rows and z
    static __host__ __device__ __forceinline__ int64_t words(int E) { return 2 * (int64_t)E + 2; }
};

template <int TYPE, int SCORE, int L, int V, bool VEC>
__global__ __launch_bounds__(kThreads) void balance_parts_kernel(BalanceArgs a, int tile, float* parts, uint32_t* tickets) {
    constexpr int GROUPS = kThreads / L;
    extern __shared__ float smem[];  // [kWaves][E] shares, [E] counts, [kWaves] rows, [kWaves] z
    float* wave_share = smem;
    int* count = reinterpret_cast<int*>(smem + kWaves * a.E);
    int* wave_rows = count + a.E;
    float* wave_z = reinterpret_cast<float*>(wave_rows + kWaves);
    const int tid = threadIdx.x, lane = tid % L, group = tid / L, wave = tid / 64;
    const int b = blockIdx.x;
    if (b == 0)
        for (int s = tid; s < a.S; s += kThreads) tickets[s] = 0;
    int row = (int)min((int64_t)b * tile, (int64_t)a.T);
    const int last = min(row + tile, a.T);
    int s = sequence_of(a.seq_offsets, row, a.S, a.T);
    while (row < last && s < a.S) {
        if (s < 0) {  // rows in front of the first sequence
            row = max(row, offset_at(a.seq_offsets, 0, a.T));
            s = 0;
            continue;
        }
        const int end = min(last, offset_at(a.seq_offsets, s + 1, a.T));
        if (end <= row) {
            ++s;
            continue;
        }
        for (int e = tid; e < a.E; e += kThreads) count[e] = 0;
        float acc[V], z = 0.0f;
        int rows = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
        if (a.logits) {
            for (int t = row + group; t < end; t += GROUPS) {
                float l[V], p[V];
                load_row<TYPE, L, V, VEC>(l, a.logits, (int64_t)t * a.stride, a.E, lane);
                mask_row<L, V, VEC>(l, a.E, lane);
                const RowSum r = shares<SCORE, L, V>(l, p);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] += p[i];
                rows += r.alive;
                z += r.lse * r.lse;
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
                if (e < a.E) wave_share[wave * a.E + e] = acc[i];
            }
            if (lane == 0) {
                wave_rows[wave] = rows;
                wave_z[wave] = z;
            }
        }
        __syncthreads();
        const int64_t id0 = (int64_t)row * a.k, ids = (int64_t)(end - row) * a.k;
        for (int64_t i = tid; i < ids; i += kThreads) {
            const int64_t e = a.topk_idx[id0 + i];
            if (e >= 0 && e < a.E) atomicAdd(&count[e], 1);
        }
        __syncthreads();
        float* out = parts + (int64_t)(b + s) * Slot::words(a.E);
        for (int e = tid; e < a.E; e += kThreads) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) v += wave_share[w * a.E + e];
            out[e] = v;
            reinterpret_cast<int*>(out)[a.E + e] = count[e];
        }
        if (tid == 0) {
            int n = 0;
            float v = 0.0f;
            for (int w = 0; w < kWaves; ++w) n += wave_rows[w], v += wave_z[w];
            reinterpret_cast<int*>(out)[2 * a.E] = n;
            out[2 * a.E + 1] = v;
        }
        __syncthreads();
        row = end;
        ++s;
    }
}

// One workgroup per sequence and kColumns experts; the last of a sequence to arrive adds up the loss.
constexpr int kColumns = 32;
__global__ __launch_bounds__(kThreads) void balance_join_kernel(BalanceArgs a, int tile, const float* parts,
                                                                uint32_t* tickets, float* sums) {
    constexpr int LANES = kThreads / kColumns;
    __shared__ float share_part[LANES][kColumns], z_part[LANES];
    __shared__ int count_part[LANES][kColumns];
    __shared__ int rows_part[LANES];
    __shared__ bool is_last;
    const int chunks = (a.E + kColumns - 1) / kColumns;
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (block >= (int64_t)chunks * a.S) return;
    const int s = (int)(block / chunks), chunk = (int)(block % chunks);
    const int col = threadIdx.x % kColumns, part = threadIdx.x / kColumns, e = chunk * kColumns + col;
    const int from = offset_at(a.seq_offsets, s, a.T), to = offset_at(a.seq_offsets, s + 1, a.T);
    const int64_t words = Slot::words(a.E);
    float share = 0.0f, z = 0.0f;
    int count = 0, rows = 0;
    if (to > from) {
        const int first = from / tile, end = (to - 1) / tile + 1;
        for (int b = first + part; b < end; b += LANES) {
            const float* in = parts + (int64_t)(b + s) * words;
            if (e < a.E) {
                share += in[e];
                count += reinterpret_cast<const int*>(in)[a.E + e];
            }
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
    float cross = 0.0f;  // counts times shares, and counts, of this workgroup's experts
    int total = 0;
    if (threadIdx.x < 64) {  // one wave, whose lanes past the columns add nothing
        share = z = 0.0f;
        count = rows = 0;
        for (int q = 0; q < LANES; ++q) {
            if (threadIdx.x < kColumns) {
                share += share_part[q][col];
                count += count_part[q][col];
            }
            rows += rows_part[q];
            z += z_part[q];
        }
        share = rows > 0 ? share / (float)rows : 0.0f;
        if (threadIdx.x < kColumns && e < a.E) {
            if (a.counts) a.counts[(int64_t)s * a.E + e] = count;
            if (a.share) a.share[(int64_t)s * a.E + e] = share;
        }
        if (chunk == 0 && threadIdx.x == 0) {
            if (a.rows) a.rows[s] = rows;
            if (a.z) a.z[s] = rows > 0 ? z / (float)rows : 0.0f;
        }
        cross = over_lanes<Sum, 64>(count > 0 ? (float)count * share : 0.0f);
        total = count;
        for (int d = 1; d < 64; d *= 2) total += __shfl_xor(total, d);
    }
    if (!a.loss) return;
    float* mine = sums + ((int64_t)s * chunks + chunk) * 2;
    if (threadIdx.x == 0) {
        __hip_atomic_store(mine, cross, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(mine + 1, __int_as_float(total), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        is_last = __hip_atomic_fetch_add(&tickets[s], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                  (uint32_t)chunks - 1;
        if (is_last) {
            const float* all = sums + (int64_t)s * chunks * 2;
            float v = 0.0f;
            int64_t n = 0;
            for (int c = 0; c < chunks; ++c) {
                v += __hip_atomic_load(all + 2 * c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                n += __float_as_int(__hip_atomic_load(all + 2 * c + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
            }
            a.loss[s] = n > 0 ? (float)a.E * v / (float)n : 0.0f;
        }
    }
}

// Rows of a tile: enough tiles to fill the GPU, and no more parts than the second kernel can add quickly.
int tile_rows(int T) {
    int tile = 16;
    while (tile < 1024 && (int64_t)tile * 512 < T) tile *= 2;
    return tile;
}

struct BalanceLayout {
    int tile, tiles;
    size_t parts = 0, tickets = 0, sums = 0, total = 0;
};
BalanceLayout balance_layout(int T, int E, int S) {
    BalanceLayout l;
    l.tile = tile_rows(T);
    l.tiles = T > 0 ? (T + l.tile - 1) / l.tile : 1;  // the first one clears the tickets
    size_t o = 0;
    auto take = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes, kAlign); return at; };
    l.parts = take((size_t)((int64_t)l.tiles + S) * Slot::words(E) * 4);
    l.tickets = take((size_t)S * 4);
    l.sums = take((size_t)S * ((E + kColumns - 1) / kColumns) * 8);
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
constexpr int kRowsPerGroup = 4;

template <int TYPE, int SCORE, int L, int V, bool VEC, int KV>
__global__ __launch_bounds__(kThreads) void gate_grad_kernel(GateGradArgs a) {
    constexpr int GROUPS = kThreads / L;
    const int lane = threadIdx.x % L;
    const int64_t first = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * GROUPS * kRowsPerGroup + threadIdx.x / L;
    int s = -2, begin = 0, end = 0;  // the sequence of the last row, and its rows
    float pull[V], zpull = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) pull[i] = 0.0f;
    for (int step = 0; step < kRowsPerGroup; ++step) {
        const int64_t t = first + (int64_t)step * GROUPS;
        if (t >= a.T) break;
        if (s == -2 || t < begin || t >= end) {
            s = sequence_of(a.seq_offsets, (int)t, a.S, a.T);
            begin = s >= 0 ? offset_at(a.seq_offsets, s, a.T) : 0;
            end = s < a.S ? offset_at(a.seq_offsets, s + 1, a.T) : a.T;
            if (s < 0 || s >= a.S) continue;
            const float n = a.rows ? (float)a.rows[s] : 0.0f;
            if (a.d_loss) {
                int64_t total = 0;
                int c[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = expert_of<L, V, VEC>(lane, i);
                    c[i] = e < a.E ? a.counts[(int64_t)s * a.E + e] : 0;
                    total += c[i];
                }
                for (int d = 1; d < L; d *= 2) total += __shfl_xor(total, d);
                const float by = n > 0.0f && total != 0 ? a.d_loss[s] / n / (float)total : 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) pull[i] = by * (float)((int64_t)c[i] * a.E - total);
            }
            zpull = a.d_z && n > 0.0f ? 2.0f * a.d_z[s] / n : 0.0f;
        }
        if (s < 0 || s >= a.S) continue;

        float l[V], p[V];
        load_row<TYPE, L, V, VEC>(l, a.logits, t * a.stride, a.E, lane);
        int id[KV];
        float lk[KV], dw[KV];
        if (a.d_topk_w) {
#pragma unroll
            for (int q = 0; q < KV; ++q) {
                const int j = lane + L * q;
                const int64_t e = j < a.k ? a.topk_idx[t * a.k + j] : -1;
                id[q] = e >= 0 && e < a.E ? (int)e : -1;
                dw[q] = id[q] >= 0 ? a.scale * a.d_topk_w[t * a.k + j] : 0.0f;
                lk[q] = id[q] >= 0 ? load1<TYPE>(a.logits, t * a.stride + id[q]) : -INFINITY;
            }
        }
        mask_row<L, V, VEC>(l, a.E, lane);
        const RowSum r = shares<SCORE, L, V>(l, p);
        float mean = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) mean += p[i] * pull[i];
        mean = over_lanes<Sum, L>(mean);
        float g[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            g[i] = p[i] * (pull[i] - mean + (SCORE == MOE_SCORE_SOFTMAX ? zpull * r.lse : 0.0f));
            if constexpr (SCORE == MOE_SCORE_SIGMOID) {
                const float x = expf(-fabsf(l[i]));
                g[i] *= (l[i] >= 0.0f ? x : 1.0f) / (1.0f + x);
            }
        }
        if (a.d_topk_w) {
            float w[KV], rest[KV];  // r and, of sigmoid scores, 1 - s
            float top = -INFINITY;
#pragma unroll
            for (int q = 0; q < KV; ++q) top = fmaxf(top, lk[q] == lk[q] ? lk[q] : INFINITY);
            if (a.renorm) top = over_lanes<Max, L>(top);
            const float by = SCORE == MOE_SCORE_SIGMOID ? (a.renorm ? fminf(top, 0.0f) : 0.0f) : a.renorm ? top : r.top;
            float sum = 0.0f;
#pragma unroll
            for (int q = 0; q < KV; ++q) {
                const bool ok = id[q] >= 0 && lk[q] != -INFINITY;
                if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
                    w[q] = ok ? expf(lk[q] - by) : 0.0f;
                    rest[q] = 1.0f;
                } else {
                    const float x = expf(-fabsf(lk[q]));
                    w[q] = ok ? (lk[q] >= 0.0f ? 1.0f : expf(lk[q] - by)) / (1.0f + x) : 0.0f;
                    rest[q] = (lk[q] >= 0.0f ? x : 1.0f) / (1.0f + x);
                }
                sum += w[q];
            }
            if (a.renorm) {
                sum = over_lanes<Sum, L>(sum);
                const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
                float m = 0.0f;
#pragma unroll
                for (int q = 0; q < KV; ++q) {
                    w[q] *= inv;
                    m += w[q] * dw[q];
                }
                m = over_lanes<Sum, L>(m);
#pragma unroll
                for (int q = 0; q < KV; ++q) w[q] *= (dw[q] - m) * rest[q];
            } else if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
                float m = 0.0f;
#pragma unroll
                for (int q = 0; q < KV; ++q) {
                    w[q] *= r.inv * dw[q];
                    m += w[q];
                }
                m = over_lanes<Sum, L>(m);
#pragma unroll
                for (int i = 0; i < V; ++i) g[i] -= p[i] * m;
            } else {
#pragma unroll
                for (int q = 0; q < KV; ++q) w[q] *= dw[q] * rest[q];
            }
            for (int j = 0; j < a.k; ++j) {  // in the order of j: an id that occurs twice adds twice
                int e = 0;
                float v = 0.0f;
#pragma unroll
                for (int q = 0; q < KV; ++q)
                    if (j / L == q) {
                        e = __shfl(id[q], j % L, L);
                        v = __shfl(w[q], j % L, L);
                    }
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (expert_of<L, V, VEC>(lane, i) == e) g[i] += v;
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (l[i] == -INFINITY) g[i] = 0.0f;
        const int64_t at = t * a.E;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const int e = 4 * (lane + L * (i / 4));
                if (e < a.E) {
                    if constexpr (TYPE == MOE_F32)
                        *reinterpret_cast<v4f*>(static_cast<float*>(a.d_logits) + at + e) =
                            v4f{g[i], g[i + 1], g[i + 2], g[i + 3]};
                    else
                        *reinterpret_cast<v2i*>(static_cast<uint16_t*>(a.d_logits) + at + e) =
                            v2i{(int)pack_bf16(g[i], g[i + 1]), (int)pack_bf16(g[i + 2], g[i + 3])};
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + L * i;
                if (e < a.E) {
                    if constexpr (TYPE == MOE_F32) static_cast<float*>(a.d_logits)[at + e] = g[i];
                    else static_cast<uint16_t*>(a.d_logits)[at + e] = (uint16_t)pack_bf16(g[i], g[i]);
                }
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
    const size_t lds = ((size_t)(kWaves + 1) * a.E + 2 * kWaves) * 4;
    hipLaunchKernelGGL((balance_parts_kernel<TYPE, SCORE, L, V, VEC>), dim3((unsigned)l.tiles), dim3(kThreads), lds, stream,
                       a, l.tile, reinterpret_cast<float*>(ws + l.parts), reinterpret_cast<uint32_t*>(ws + l.tickets));
}
template <int TYPE, int SCORE, int L, int V, bool VEC, int KV>
void grad_go(const GateGradArgs& a, hipStream_t stream) {
    const int rows = kThreads / L * kRowsPerGroup;
    hipLaunchKernelGGL((gate_grad_kernel<TYPE, SCORE, L, V, VEC, KV>), wide_grid(((int64_t)a.T + rows - 1) / rows),
                       dim3(kThreads), 0, stream, a);
}

// f(type, score, lanes, values, vector loads, chosen ids per lane) as compile-time constants
template <int N>
using Int = std::integral_constant<int, N>;
template <class F>
void with_lanes(int E, F f) {
    if (E <= 32) f(Int<8>{}, Int<4>{}, Int<4>{});
    else if (E <= 64) f(Int<16>{}, Int<4>{}, Int<4>{});
    else if (E <= 128) f(Int<32>{}, Int<4>{}, Int<2>{});
    else if (E <= 256) f(Int<64>{}, Int<4>{}, Int<1>{});
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
    const int chunks = (a.E + kColumns - 1) / kColumns;
    hipLaunchKernelGGL(balance_join_kernel, wide_grid((int64_t)chunks * a.S), dim3(kThreads), 0, stream, a, l.tile,
                       reinterpret_cast<const float*>(base + l.parts), reinterpret_cast<uint32_t*>(base + l.tickets),
                       reinterpret_cast<float*>(base + l.sums));
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
