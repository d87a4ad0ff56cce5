// Gate: scores, group choice, top-k and weights of one row of router logits per token.
//
// Definition (exact_row): every comparison that decides an order is made on a 64-bit key that rises with the
// order value (FP64, or the logit itself without a bias), with NaN on top and 0 for what may not be chosen;
// equal keys go to the lowest expert.
//
// gate_kernel finds the same answer in 32 bits and proves it, row by row.  It takes the k + 2 best by 32-bit
// keys that hold a shortened order value and the expert's index, ranks those among each other on the values
// themselves (FP64), and checks that the next key is too small to belong among the first k, its shortening
// and the error of FP32 scores allowed for.  Marks of groups too close for FP32 are formed again in FP64.  A row that
// fails (three candidates within the error, marks of softmax scores within theirs, a NaN, a spread that the keys
// cannot hold) is done again by exact_row, which adds 5.5 us to a call of 128.
// How many do depends on how far the k + 1st candidate is from the rest.  Of 262,144 rows of 256 experts, top 8, logits
// N(0, 1): none without a bias, none of sigmoid scores, 10 of softmax scores under a bias of 201 steps of 0.001.  A call
// of 65536 rows (18 to 31 us) takes up to 190 where nearly all rows fail, as rows do of equal FP32 logits without a bias
// (147), of softmax scores with one logit of 16 and a bias of few distinct values (162; of 201 values 31, none fails),
// and of sigmoid scores of N(0, 10), saturated, with a zero bias (147, 190 in groups).
//
// Bound by instructions, not by memory: 16 lanes share a row (four rows a wave; 64 lanes for long rows), a
// lane keeps its D largest keys sorted, and a round of the selection is four DPP maxima and D moves for all
// rows of the wave.  Packing the index into the key makes a comparison of two candidates one instruction.
// 65536 x 384, top 6, no bias: 24 us FP32 (106 MB, 4.4 TB/s), 20.5 BF16 (56 MB); with a bias 28 to 32.  16384 x 256,
// top 8: 7.7 without a bias, 9 with one, 10.7 with 8 groups marked by pairs; 128 such rows 5.1, where a kernel
// that stores one word takes 3.7 of launch.
#include "moe_internal.h"

#include <cfloat>

namespace moe {
namespace {

constexpr int kWaves = 4;

// Rising with v as numbers compare (-0 and +0 alike), NaN above everything; never 0.
__device__ __forceinline__ uint64_t order_key(double v) {
    if (v != v) return ~0ull;
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return b & (1ull << 63) ? ~b : b | (1ull << 63);
}

// ---- moves between lanes: DPP inside a row of 16, swaps of rows and halves above

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kXor7 = 0x141, kXor15 = 0x140, kRor1 = 0x121;  // kRor1: around the row

__device__ __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }
__device__ __forceinline__ float real(uint32_t v) { return __uint_as_float(v); }

// op over L = 2 .. 64 neighbouring lanes (a run-time power of two), in all of them.
template <class Op>
__device__ __forceinline__ uint32_t across(uint32_t v, int L, Op op) {
    if (L > 1) v = op(v, dpp<kXor1>(v));
    if (L > 2) v = op(v, dpp<kXor2>(v));
    if (L > 4) v = op(v, dpp<kXor7>(v));
    if (L > 8) v = op(v, dpp<kXor15>(v));
    if (L > 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = op(r[0], r[1]);
    }
    if (L > 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = op(r[0], r[1]);
    }
    return v;
}
struct MaxU {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return max(a, b); }
};
struct MaxF {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return bits(fmaxf(real(a), real(b))); }
};
struct MinF {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return bits(fminf(real(a), real(b))); }
};
struct AddF {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return bits(real(a) + real(b)); }
};
struct AddU {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a + b; }
};
struct MinU {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return min(a, b); }
};
__device__ __forceinline__ uint64_t join(uint32_t hi, uint32_t lo) { return ((uint64_t)hi << 32) | lo; }
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double((long long)join(dpp<CTRL>((uint32_t)(b >> 32)), dpp<CTRL>((uint32_t)b)));
}
// op over the wave on 64-bit values, in all lanes.
template <class Op>
__device__ __forceinline__ uint64_t across64(uint64_t v, Op op) {
    auto two = [&](uint32_t hi, uint32_t lo) { v = op(v, join(hi, lo)); };
    two(dpp<kXor1>((uint32_t)(v >> 32)), dpp<kXor1>((uint32_t)v));
    two(dpp<kXor2>((uint32_t)(v >> 32)), dpp<kXor2>((uint32_t)v));
    two(dpp<kXor7>((uint32_t)(v >> 32)), dpp<kXor7>((uint32_t)v));
    two(dpp<kXor15>((uint32_t)(v >> 32)), dpp<kXor15>((uint32_t)v));
    {
        const uint32_t hi = (uint32_t)(v >> 32), lo = (uint32_t)v;
        const auto h = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
        const auto l = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
        v = op(join(h[0], l[0]), join(h[1], l[1]));
    }
    const uint32_t hi = (uint32_t)(v >> 32), lo = (uint32_t)v;
    const auto h = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
    const auto l = __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
    return op(join(h[0], l[0]), join(h[1], l[1]));
}

__device__ __forceinline__ double wave_max(double v) {
    const auto op = [](uint64_t a, uint64_t b) {
        return (uint64_t)__double_as_longlong(fmax(__longlong_as_double((long long)a), __longlong_as_double((long long)b)));
    };
    return __longlong_as_double((long long)across64((uint64_t)__double_as_longlong(v), op));
}
__device__ __forceinline__ double wave_sum(double v) {
    const auto op = [](uint64_t a, uint64_t b) {
        return (uint64_t)__double_as_longlong(__longlong_as_double((long long)a) + __longlong_as_double((long long)b));
    };
    return __longlong_as_double((long long)across64((uint64_t)__double_as_longlong(v), op));
}
__device__ __forceinline__ float load_logit(const GateArgs& a, int64_t i) {
    if (a.logits_type == MOE_F32) return static_cast<const float*>(a.logits)[i];
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[i] << 16);
}
// The number that order_key maps to key (its NaN for ~0).
__device__ __forceinline__ double order_value(uint64_t key) {
    return __longlong_as_double((long long)(key >> 63 ? key & ~(1ull << 63) : ~key));
}

// One row by one wave, with every score in FP64; lane l takes experts l, l + 64, ...  keys: E words of LDS of
// this wave.  Rolled loops and keys in LDS: the function is called from gate_kernel for few rows, whose
// registers it must not multiply.
typedef __attribute__((address_space(3))) uint64_t lds_u64;
__device__ __forceinline__ void exact_row(const GateArgs& a, int64_t t, lds_u64* keys) {
    const int lane = threadIdx.x & 63;
    const bool soft = a.score == MOE_SCORE_SOFTMAX;
    auto logit = [&](int e) { return (double)load_logit(a, t * a.stride + e); };
    double top = -INFINITY, sum = 0.0;
    if (soft) {
        bool nan = false;
        for (int e = lane; e < a.E; e += 64) {
            const double l = logit(e);
            nan |= l != l;
            top = fmax(top, l);
        }
        top = __any(nan) ? NAN : wave_max(top);
        for (int e = lane; e < a.E; e += 64) {
            const double l = logit(e);
            sum += l == -INFINITY ? 0.0 : exp(l - top);
        }
        sum = wave_sum(sum);
    }
    auto score = [&](double l) { return soft ? exp(l - top) / sum : 1.0 / (1.0 + exp(-l)); };
    // four at a time, so that their loads are in flight together
    for (int base = lane; base < a.E; base += 256) {
        float l[4], b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int e = min(base + 64 * u, a.E - 1);
            l[u] = load_logit(a, t * a.stride + e);
            b[u] = a.bias ? a.bias[e] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int e = base + 64 * u;
            double c = (double)l[u];
            if (a.bias && l[u] != -INFINITY) c = score(c) + (double)b[u];
            if (e < a.E) keys[e] = c == -INFINITY ? 0 : order_key(c);
        }
    }
    if (a.groups > 1) {
        // 64 / groups lanes, to a power of two, for each group: its two largest keys in all of them
        const int n = a.E / a.groups;
        int lpg = 64;
        while (lpg * a.groups > 64) lpg /= 2;
        const int group = lane / lpg;
        const bool pair = a.group_score == MOE_GROUP_TOP2;
        __builtin_amdgcn_wave_barrier();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // other lanes' keys are read from here on
        uint64_t k1 = 0, k2 = 0;
        auto with = [&](uint64_t o1, uint64_t o2) {
            const uint64_t low = min(k1, o1);
            k1 = max(k1, o1);
            k2 = max(low, max(k2, o2));
        };
        if (group < a.groups)
            for (int e = lane & (lpg - 1); e < n; e += lpg) with(keys[group * n + e], 0);
        for (int s = 1; s < lpg; s *= 2)
            with((uint64_t)__shfl_xor((unsigned long long)k1, s), (uint64_t)__shfl_xor((unsigned long long)k2, s));
        uint64_t mark = k1;
        if (pair && k1 != 0) {  // without a bias the keys are those of the logits, and scores rise with them
            double v = order_value(k1), w = k2 ? order_value(k2) : 0.0;
            if (!a.bias) {
                v = score(v);
                w = k2 ? score(w) : 0.0;
            }
            mark = order_key(v + w);
        }
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const uint64_t o = (uint64_t)__shfl((unsigned long long)mark, g * lpg);
            rank += (o > mark) | ((o == mark) & (g < group));
        }
        const bool kept = (rank < a.topk_groups) & (group < a.groups);
        if (!kept && group < a.groups)
            for (int e = lane & (lpg - 1); e < n; e += lpg) keys[group * n + e] = 0;
        __builtin_amdgcn_wave_barrier();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    // Lane j keeps the j-th choice.  A lane knows its own largest key, and looks for the next when that is taken; the
    // high halves of the lanes' keys decide unless two are equal (0.31 us a choice; 0.37 with the whole keys and
    // all lanes' indices compared).
    uint32_t hi, lo;
    int at;
    auto own_best = [&] {
        uint64_t k = 0;
        at = 0;
#pragma unroll 4
        for (int e = lane; e < a.E; e += 64) {
            const uint64_t o = keys[e];
            at = o > k ? e : at;
            k = max(k, o);
        }
        hi = (uint32_t)(k >> 32);
        lo = (uint32_t)k;
    };
    own_best();
    int mine = -1;
    for (int j = 0; j < a.k; ++j) {
        const uint32_t top_hi = across(hi, 64, MaxU{});
        if (top_hi == 0) break;  // no candidate's
        uint64_t who = __ballot(hi == top_hi);
        if (who & (who - 1)) {
            const uint32_t top_lo = across(hi == top_hi ? lo : 0, 64, MaxU{});
            const bool same = (hi == top_hi) & (lo == top_lo);
            const uint32_t first = across(same ? (uint32_t)at : ~0u, 64, MinU{});
            who = __ballot(same & ((uint32_t)at == first));
        }
        const int winner = __ffsll((long long)who) - 1, taken = __builtin_amdgcn_readlane(at, winner);
        if (lane == j) mine = taken;
        if (lane == winner) {
            keys[at] = 0;
            own_best();
        }
    }
    double w = mine >= 0 ? score(logit(mine)) : 0.0;
    if (a.renorm) {
        const double total = wave_sum(w);
        w = total == 0.0 ? 0.0 : w / total;
    }
    if (lane < a.k) {
        a.topk_idx[t * a.k + lane] = mine;
        a.topk_w[t * a.k + lane] = (float)(mine < 0 ? 0.0 : w * (double)a.scale);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // before the next row's keys
}

// ---- 32 bits with proof

// Keys in falling order.
__device__ __forceinline__ void order(uint32_t& a, uint32_t& b) {
    const uint32_t hi = max(a, b);
    b = min(a, b);
    a = hi;
}
// Odd-even merge sort of k[LO .. LO + N), by recursion that the compiler has to unroll.
template <int LO, int N, int R, int SIZE>
__device__ __forceinline__ void merge_halves(uint32_t (&k)[SIZE]) {
    if constexpr (2 * R < N) {
        merge_halves<LO, N, 2 * R>(k);
        merge_halves<LO + R, N, 2 * R>(k);
#pragma unroll
        for (int i = LO + R; i + R < LO + N; i += 2 * R) order(k[i], k[i + R]);
    } else {
        order(k[LO], k[LO + R]);
    }
}
template <int LO, int N, int SIZE>
__device__ __forceinline__ void sort(uint32_t (&k)[SIZE]) {
    if constexpr (N > 1) {
        sort<LO, N / 2>(k);
        sort<LO + N / 2, N / 2>(k);
        merge_halves<LO, N, 1>(k);
    }
}
template <int N>
__device__ __forceinline__ void merge(uint32_t (&top)[N], const uint32_t (&more)[N]) {  // both sorted
#pragma unroll
    for (int i = 0; i < N; ++i) top[i] = max(top[i], more[N - 1 - i]);  // bitonic
#pragma unroll
    for (int q = N / 2; q >= 1; q /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if ((i & q) == 0) order(top[i], top[i + q]);
}

// 1 / (1 + e^-l) with the hardware's 2^x and reciprocal: within 2^-22 (the argument's rounding moves it by
// at most |l| s (1 - s) 2^-24 < 2^-25, the exponential, the sum and the reciprocal by one unit each).
__device__ __forceinline__ float sigmoid32(float l) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l * -1.44269504088896341f));
}
__device__ __forceinline__ float exp32(float d) { return __builtin_amdgcn_exp2f(d * 1.44269504088896341f); }
// e^d for d <= 0 within 3 * 2^-24 of it: 2^(the product as rounded) by the hardware (2), times 1 + ln 2 times what
// that rounding and the constant's left out (1).
__device__ __forceinline__ float exp_whole(float d) {
    const float t = d * 1.44269504088896341f;
    const float rest = fmaf(d, 1.44269504088896341f, -t) + d * 1.92596299e-8f;
    const float e = __builtin_amdgcn_exp2f(t);
    return t < -200.0f ? 0.0f : fmaf(e, rest * 0.693147182f, e);
}

constexpr int kKeyRange = 4;  // order values from a row's largest down to this far below it have keys of their own

// Rows of up to L * V experts, k <= 16.  n: experts per group; 1 << lpg_shift lanes per group, groups of them
// at most L (one group: all lanes).  A lane takes every (1 << lpg_shift)-th expert of its group, or with vec
// (groups, rows and bias start on 4 elements) run of 4.  index_bits hold every place that a lane can name.
struct GateFast {
    GateArgs a;
    int n, lpg_shift, index_bits;
    bool vec;
};

template <int L, int V, int D>
__global__ __launch_bounds__(64 * kWaves) void gate_kernel(GateFast f) {
    constexpr int ROWS = 64 / L, EXPERTS = L * V < kMaxGateExperts ? L * V : kMaxGateExperts;
    __shared__ uint64_t keys[kWaves][EXPERTS];
    const GateArgs& a = f.a;
    const int lane = threadIdx.x & 63, sub = lane & (L - 1);
    const int64_t t0 = (((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kWaves + threadIdx.x / 64) * ROWS;
    if (t0 >= a.T) return;
    const int64_t t = min(t0 + lane / L, (int64_t)a.T - 1);  // lanes past the last row repeat it, and store nothing
    const bool soft = a.score == MOE_SCORE_SOFTMAX, grouped = a.groups > 1, biased = a.bias != nullptr;
    const bool pair = grouped && a.group_score == MOE_GROUP_TOP2;
    const int lpg = 1 << f.lpg_shift, group = sub >> f.lpg_shift;
    // the first `held` of the lane's experts are inside its group
    const int shift = f.vec ? f.lpg_shift + 2 : f.lpg_shift, step = 1 << shift;
    const int member = (sub & (lpg - 1)) << (f.vec ? 2 : 0);
    const int e0 = group * f.n + member;
    const int own = max(f.n - member + step - 1, 0) >> shift;
    const int held = group < a.groups ? own << (f.vec ? 2 : 0) : 0;
    const int by1 = f.vec ? 1 : step, by4 = f.vec ? step : 4 * step;
    auto expert = [&](int i) { return e0 + by4 * (i / 4) + by1 * (i % 4); };

    float c[V];  // the logits, then the order values; -infinity: may not be chosen
    const int64_t row = t * a.stride;
    if (a.logits_type == MOE_F32) {
        const float* p = static_cast<const float*>(a.logits) + row;
        if (f.vec) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(p + min(e0 + step * (i / 4), a.E - 4));
                c[i] = v.x; c[i + 1] = v.y; c[i + 2] = v.z; c[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) c[i] = p[min(e0 + step * i, a.E - 1)];
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(a.logits) + row;
        if (f.vec) {
            uint2 v[V / 4];
#pragma unroll
            for (int i = 0; i < V; i += 4)
                v[i / 4] = *reinterpret_cast<const uint2*>(p + min(e0 + step * (i / 4), a.E - 4));
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                c[i] = real(v[i / 4].x << 16); c[i + 1] = real(v[i / 4].x & 0xFFFF0000u);
                c[i + 2] = real(v[i / 4].y << 16); c[i + 3] = real(v[i / 4].y & 0xFFFF0000u);
            }
        } else {
            uint16_t v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = p[min(e0 + step * i, a.E - 1)];
#pragma unroll
            for (int i = 0; i < V; ++i) c[i] = real((uint32_t)v[i] << 16);
        }
    }
    if (!__all(held >= V)) {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = i < held ? c[i] : -INFINITY;
    }
    bool doubt = false;  // of this lane's row
    float top = -INFINITY;
    // Softmax in units of 2^-24: an argument is d = top - l, off by 1 unit times d (by 3 with exp32's product),
    // and the mean of d under the softmax's own weights is at most ln 1024 < 7.  A sum that divides scores is off
    // by 7 + 3 (exp_whole) and added in FP64, one that only marks groups by 21 + 1 + 22 (additions).  An FP32 score
    // is e^-d <= 1 times inv, the largest score: off by at most 53 (d e^-d < 0.37) times inv.  (Exponentials in FP64
    // would be V a lane, where the picks take one; weights of a sum off by 10 are within 11 of the formula's.)
    float sum = 0.0f, inv = 0.0f;
    double sum64 = 0.0;
    if (soft) {
#pragma unroll
        for (int i = 0; i < V; ++i) top = fmaxf(top, c[i]);
        top = real(across(bits(top), L, MaxF{}));
        doubt |= top == INFINITY;
        top = top == -INFINITY ? 0.0f : top;
        if (biased || !a.renorm) {
#pragma unroll
            for (int i = 0; i < V; ++i) sum64 += (double)exp_whole(c[i] - top);
            if constexpr (L == 64) {
                sum64 = wave_sum(sum64);
            } else {
                sum64 += dpp_f64<kXor1>(sum64);
                sum64 += dpp_f64<kXor2>(sum64);
                sum64 += dpp_f64<kXor7>(sum64);
                sum64 += dpp_f64<kXor15>(sum64);
            }
            sum = (float)sum64;
        } else if (pair) {
#pragma unroll
            for (int i = 0; i < V; ++i) sum += exp32(c[i] - top);
            sum = real(across(bits(sum), L, AddF{}));
        }
        inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    }
    const float err = soft ? 0x1p-18f * inv : 0x1p-22f;  // at least that of an FP32 score
    auto to_scores = [&](float(&v)[V]) {           // of -infinity: 0
        if (soft) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = exp32(v[i] - top) * inv;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = sigmoid32(v[i]);
        }
    };
    if (biased) {
        float b[V];
        if (f.vec) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(a.bias + min(e0 + step * (i / 4), a.E - 4));
                b[i] = v.x; b[i + 1] = v.y; b[i + 2] = v.z; b[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) b[i] = a.bias[min(e0 + step * i, a.E - 1)];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) b[i] = c[i] == -INFINITY ? -INFINITY : b[i];
        to_scores(c);
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] += b[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) doubt |= c[i] != c[i];
    if (grouped) {
        // the two largest of the group
        float m1 = -INFINITY, m2 = -INFINITY;
        auto most_of = [&](const float(&v)[V]) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                m2 = fmaxf(m2, fminf(m1, v[i]));
                m1 = fmaxf(m1, v[i]);
            }
        };
        most_of(c);
        auto with = [&](float o1, float o2) {
            m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
            m1 = fmaxf(m1, o1);
        };
        if (lpg > 1) with(real(dpp<kXor1>(bits(m1))), real(dpp<kXor1>(bits(m2))));
        if (lpg > 2) with(real(dpp<kXor2>(bits(m1))), real(dpp<kXor2>(bits(m2))));
        if (lpg > 4) with(real(dpp<kXor7>(bits(m1))), real(dpp<kXor7>(bits(m2))));
        if (lpg > 8) with(real(dpp<kXor15>(bits(m1))), real(dpp<kXor15>(bits(m2))));
        if (lpg > 16) with(__shfl_xor(m1, 16), __shfl_xor(m2, 16));
        const float least = pair ? m2 : m1;  // what counts for the mark is no lower
        if (pair && !biased) {  // scores rise with the logits
            m1 = m1 == -INFINITY ? m1 : soft ? exp32(m1 - top) * inv : sigmoid32(m1);
            m2 = m2 == -INFINITY ? m2 : soft ? exp32(m2 - top) * inv : sigmoid32(m2);
        }
        const float mark = pair && m2 > -INFINITY ? m1 + m2 : m1;
        doubt |= (m2 > -INFINITY) & (mark == -INFINITY);  // a sum beyond FP32, that ranks with a group of no candidate
        int rank = 0;
        for (int g0 = 0; g0 < a.groups; g0 += 4) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int g = g0 + u;
                const float o = __shfl(mark, g << f.lpg_shift, L);  // past the last group: not counted
                rank += (g < a.groups) & ((o > mark) | ((o == mark) & (g < group)));
            }
        }
        bool kept = (rank < a.topk_groups) & (group < a.groups);
        // logits compare exactly; sums of scores have to differ by more than the errors of both
        if (pair || biased) {
            const float low = real(across(bits((kept & (mark > -INFINITY)) ? mark : INFINITY), L, MinF{}));
            const float high = real(across(bits(kept ? -INFINITY : mark), L, MaxF{}));
            const float size = fmaxf(m1 > -INFINITY ? fabsf(m1) : 0.0f, m2 > -INFINITY ? fabsf(m2) : 0.0f);
            const float amp = real(across(bits(size), L, MaxF{}));  // four c and two sums, each rounded to 2^-24
            const float slack = 4.0f * err + 0x1p-21f * amp;
            const bool close = (high > -INFINITY) & !(low - high > slack);
            doubt |= close & (soft | !(amp < INFINITY));
            if (!soft && __any(close)) {
                // The marks again in FP64, as exact_row forms them, from the experts that may be the group's
                // largest.  (4 of 100,000 random rows of 256 experts in 8 groups; 16384 such rows, of which some
                // are among them, 11.0 us, 12.5 to 14 with the rows done again.)
                const float from = biased ? least - slack : least;
                uint32_t may = 0;
#pragma unroll
                for (int i = 0; i < V; ++i) may |= ((c[i] >= from) & (c[i] > -INFINITY)) ? 1u << i : 0;
                double x1 = -INFINITY, x2 = -INFINITY;
                auto add = [&](double o1, double o2) {
                    x2 = fmax(fmin(x1, o1), fmax(x2, o2));
                    x1 = fmax(x1, o1);
                };
                while (__any(may != 0)) {
                    if (may) {
                        const int e = expert(__ffs((int)may) - 1);
                        double v = (double)load_logit(a, row + e);
                        if (pair || biased) v = 1.0 / (1.0 + exp(-v));
                        if (biased) v += (double)a.bias[e];
                        add(v, -INFINITY);
                    }
                    may &= may - 1;
                }
                for (int r = 1; r < lpg; r *= 2) add(__shfl_xor(x1, r), __shfl_xor(x2, r));
                const double exact = pair && x2 > -INFINITY ? x1 + x2 : x1;
                rank = 0;
                for (int g = 0; g < a.groups; ++g) {
                    const double o = __shfl(exact, g << f.lpg_shift, L);
                    rank += (o > exact) | ((o == exact) & (g < group));
                }
                kept = (rank < a.topk_groups) & (group < a.groups);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = kept ? c[i] : -INFINITY;
    }

    // The proposal.  Without a bias a key's value is the logit's bits, rising with it, less the lowest
    // index_bits; with one it counts steps of kKeyRange 2^(index_bits - 32) from the bottom of the range.
    // Keys below `none` are no candidates.
    const uint32_t mask = (1u << f.index_bits) - 1;
    uint32_t best[V], none;
    float scale = 0.0f, base = 0.0f;
    if (biased) {
        float hi = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) hi = fmaxf(hi, c[i]);
        // From -2^100 down, and where there is no candidate, the range stays where it is, so that base is below infinity:
        // candidates below the range get no keys, and the row is done again.  (With base = +infinity all keys were the
        // range's upper end, in order of the index, and those of places past the row's end NaN.)  base is -infinity
        // under a huge hi; then an infinite c makes a NaN, at either end: that is an expert, and the row in doubt.
        hi = fmaxf(real(across(bits(hi), L, MaxF{})), -0x1p100f);
        const float steps = (float)(1u << (32 - f.index_bits));
        scale = steps / kKeyRange;
        base = (steps - 8.0f) - hi * scale;  // hi goes to steps - 8, a few up or down by rounding
        none = 1u << f.index_bits;
#pragma unroll
        for (int i = 0; i < V; ++i) {  // base < infinity: what may not be chosen goes to 0, also where nothing may
            const float v = __builtin_amdgcn_fmed3f(fmaf(c[i], scale, base), 0.0f, steps - 1.0f);
            best[i] = ((uint32_t)v << f.index_bits) | (mask - expert(i));
        }
    } else {
        none = 0x00800000u;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t b = bits(c[i] + 0.0f);  // -0 to +0
            const uint32_t o = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
            best[i] = (o & ~mask) | (mask - expert(i));
        }
    }
    uint32_t lead[D];
#pragma unroll
    for (int j = 0; j < V; j += D) {
        uint32_t more[D];
#pragma unroll
        for (int i = 0; i < D; ++i) more[i] = best[j + i];
        sort<0, D>(more);
        if (j == 0) {
#pragma unroll
            for (int i = 0; i < D; ++i) lead[i] = more[i];
        } else {
            merge<D>(lead, more);
        }
    }
    const int picks = min(a.k + 2, 16);
    uint32_t mine = 0;  // lane j of the row keeps the j-th
    for (int j = 0; j < picks; ++j) {
        const uint32_t w = across(lead[0], L, MaxU{});
        // the lane that had it moves up by one; as masks, for a choice of array elements becomes one of indices
        const uint32_t up = lead[0] == w ? ~0u : 0u;
#pragma unroll
        for (int d = 0; d + 1 < D; ++d) lead[d] = (lead[d] & ~up) | (lead[d + 1] & up);
        lead[D - 1] &= ~up;
        if (sub == j) mine = w;
    }
    // what is left is at most the largest key left, unless a lane gave all that its list held
    const uint32_t left = across(lead[0], L, MaxU{}) >> f.index_bits;
    if (D < V) doubt |= lead[0] == 0;

    // The picks' scores in FP64 (one exponential per lane serves all of the wave's rows), their order values
    // and ranks.  The error of a softmax's sum (10 units) moves two scores apart or together by that part of
    // their difference: their order values under a bias have to differ by more, the 64-bit roundings of both
    // allowed for, or score and bias be the same.
    const bool picked = (sub < picks) & (mine >= none);
    const int id = picked ? (int)(mask - (mine & mask)) : 1 << 30;
    const float l = picked ? load_logit(a, t * a.stride + id) : -INFINITY;
    const float b = (picked & biased) ? a.bias[id] : 0.0f;
    const double e = exp(soft ? (double)l - (double)top : -(double)l);
    double s = soft ? e : 1.0 / (1.0 + e);
    if (soft && (biased || !a.renorm)) s = sum64 > 0.0 ? s / sum64 : 0.0;
    const double value = !picked ? -INFINITY : biased ? s + (double)b : (double)l;
    const float gap = biased ? 2.0f * err + 0x1p-22f * fabsf((float)value) : 0.0f;
    // The picks come in the order of their keys, which is nearly always that of their values: one comparison with
    // the pick before then says that of all.  Under a softmax and a bias neighbours that are apart by the error of
    // the largest score's part say it of all pairs.
    int rank = sub;
    double o = dpp_f64<kRor1>(value);  // of the lane before
    uint32_t oid = dpp<kRor1>((uint32_t)id);
    const bool weighed = soft && biased;  // order values that the sum's error moves
    const bool sorted = weighed ? o - value > (double)inv * 0x1.1p-20 + (fabs(o) + fabs(value)) * 0x1p-51
                                : (o > value) | ((o == value) & ((int)oid < id));
    if (__any(picked & (sub > 0) & !sorted)) {
        double os = dpp_f64<kRor1>(s);
        uint32_t ob = dpp<kRor1>(bits(b));
        rank = 0;
        for (int r = 1; r < 16; ++r) {  // all pairs of the row of 16 lanes that holds the picks
            rank += (o > value) | ((o == value) & ((int)oid < id));
            const bool near = fabs(o - value) <= fabs(os - s) * 0x1p-20 + fabs(value) * 0x1p-51;
            doubt |= weighed & picked & near & ((os != s) | (real(ob) != b));  // lanes without a pick: infinitely far
            o = dpp_f64<kRor1>(o);
            oid = dpp<kRor1>(oid);
            os = dpp_f64<kRor1>(os);
            ob = dpp<kRor1>(ob);
        }
    }
    const bool chosen = picked & (rank < a.k);

    // No other candidate reaches the last choice.
    const uint64_t row_lanes = L == 64 ? ~0ull : ((1ull << (L & 63)) - 1) << (lane & ~(L - 1));
    const int n_chosen = __popcll(__ballot(chosen) & row_lanes);
    const bool last = picked & (rank == a.k - 1);
    if (biased) {
        // in steps of the keys: one that the key cuts off and one for the rounding of each side
        doubt |= last & !((float)left + 3.0f < fmaf((float)value - gap, scale, base));
        if (__any(n_chosen < a.k)) {  // every candidate has to be a choice, those below the keys' range too
            int count = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) count += c[i] > -INFINITY;
            doubt |= (n_chosen < a.k) & ((int)across((uint32_t)count, L, AddU{}) != n_chosen);
        }
    } else {
        // keys of BF16 logits hold them whole, and order equal ones by their index
        doubt |= last & (a.logits_type == MOE_F32) & (left >= mine >> f.index_bits);
    }

    s = chosen ? s : 0.0;
    if (a.renorm) {
        double total = s;  // the choices lie in one DPP row
        total += dpp_f64<kXor1>(total);
        total += dpp_f64<kXor2>(total);
        total += dpp_f64<kXor7>(total);
        total += dpp_f64<kXor15>(total);
        s = total == 0.0 ? 0.0 : s / total;
    }
    const uint64_t doubts = __ballot(doubt);
    if ((sub < 16) & (t0 + lane / L < a.T) & !(doubts & row_lanes)) {
        if (chosen) {
            a.topk_idx[t * a.k + rank] = id;
            a.topk_w[t * a.k + rank] = (float)(s * (double)a.scale);
        }
        if ((sub >= n_chosen) & (sub < a.k)) {  // the choices that there are not
            a.topk_idx[t * a.k + sub] = -1;
            a.topk_w[t * a.k + sub] = 0.0f;
        }
    }
    if (doubts)
        for (int r = 0; r < ROWS && t0 + r < a.T; ++r)
            if (doubts >> (r * L) & (~0ull >> (64 - L))) exact_row(a, t0 + r, (lds_u64*)keys[threadIdx.x / 64]);
}

// Rows of more than 16 choices.
__global__ __launch_bounds__(64 * kWaves) void gate_exact_kernel(GateArgs a) {
    __shared__ uint64_t keys[kWaves][kMaxGateExperts];
    const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kWaves + threadIdx.x / 64;
    if (t < a.T) exact_row(a, t, (lds_u64*)keys[threadIdx.x / 64]);
}

hipError_t launch_exact(const GateArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(gate_exact_kernel, wide_grid(((int64_t)a.T + kWaves - 1) / kWaves), dim3(64 * kWaves), 0, stream, a);
    return hipGetLastError();
}

template <int L, int V, int D>
hipError_t launch(const GateFast& f, hipStream_t stream) {
    constexpr int ROWS = kWaves * (64 / L);
    hipLaunchKernelGGL((gate_kernel<L, V, D>), wide_grid(((int64_t)f.a.T + ROWS - 1) / ROWS), dim3(64 * kWaves), 0, stream, f);
    return hipGetLastError();
}

}  // namespace

GateChoice choose_gate(const GateArgs& a) {
    GateChoice c{};
    c.lanes = 64;
    if (a.k > 16) return c;
    int padded = 1;  // groups to a power of two
    while (padded < a.groups) padded *= 2;
    const int n = a.E / a.groups;
    // 16 lanes a row while a lane then holds at most 32 experts, else 64
    auto lanes_hold = [&](int L) { return padded > L ? 1 << 20 : (n + L / padded - 1) / (L / padded); };
    if (lanes_hold(16) <= 32) c.lanes = 16;
    c.lpg = c.lanes / padded;
    const int64_t size = a.logits_type == MOE_F32 ? 4 : 2;
    c.vec = n % 4 == 0 && a.stride % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % (4 * size) == 0 &&
            reinterpret_cast<uintptr_t>(a.bias) % 16 == 0 && (n / 4 + c.lpg - 1) / c.lpg * 4 <= 32;
    const int hold = c.vec ? (n / 4 + c.lpg - 1) / c.lpg * 4 : lanes_hold(c.lanes);
    // 4, 8, 16, 24 or 32 experts a lane; 24 for lists of 8 keys only, which divide it (65536 x 384, top 6, bias: 29.3 us,
    // 36.2 with 32; BF16 without a bias 19.8, 25.7; 128 rows 4.5, 5.3), and
    // for 16 lanes (at 64 it was not tried)
    c.values = 4;
    while (c.values < hold)
        c.values += c.values == 16 && c.lanes == 16 && a.k <= 8 ? 8 : c.values == 24 ? 8 : c.values;
    if (c.lanes == 64 && c.values < 16) c.values = 16;
    c.list = std::min(c.values, a.k > 8 ? 16 : 8);
    c.index_bits = 8;  // at least: FP32 counts the keys' steps, 2^(32 - index_bits) of them, one by one to 2^24
    while ((1 << c.index_bits) < (padded - 1) * n + c.lpg * c.values) ++c.index_bits;
    return c;
}

hipError_t launch_gate(const GateArgs& a, hipStream_t stream) {
    const GateChoice c = choose_gate(a);
    if (c.values == 0) return launch_exact(a, stream);
    const GateFast f{a, a.E / a.groups, __builtin_ctz(c.lpg), c.index_bits, c.vec};
    if (c.lanes == 16) {
        if (c.values == 4) return launch<16, 4, 4>(f, stream);
        if (c.values == 8) return launch<16, 8, 8>(f, stream);
        if (c.list == 16) return c.values == 16 ? launch<16, 16, 16>(f, stream) : launch<16, 32, 16>(f, stream);
        if (c.values == 16) return launch<16, 16, 8>(f, stream);
        return c.values == 24 ? launch<16, 24, 8>(f, stream) : launch<16, 32, 8>(f, stream);
    }
    if (c.list == 16) return c.values == 16 ? launch<64, 16, 16>(f, stream) : launch<64, 32, 16>(f, stream);
    return c.values == 16 ? launch<64, 16, 8>(f, stream) : launch<64, 32, 8>(f, stream);
}

}  // namespace moe
