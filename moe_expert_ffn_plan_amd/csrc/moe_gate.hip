// Gate: scores, group choice, top-k and weights of one row of router logits per token.
//
// One wave per token; lane l holds experts l, l + 64, ...  Every comparison that decides an order is made
// on a 64-bit key that rises with the order value (FP64, or the logit itself without a bias), with NaN on
// top and 0 for what may not be chosen; equal keys go to the lowest expert.
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kWaves = 4;

// Rising with v as numbers compare (-0 and +0 alike), NaN above everything; never 0.
__device__ __forceinline__ uint64_t order_key(double v) {
    if (v != v) return ~0ull;
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return b & (1ull << 63) ? ~b : b | (1ull << 63);
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int m) {
    return (uint64_t)__shfl_xor((unsigned long long)v, m);
}
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
    for (int s = 1; s < 64; s *= 2) v = fmax(v, __shfl_xor(v, s));
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int s = 1; s < 64; s *= 2) v += __shfl_xor(v, s);
    return v;
}
// The largest key of the wave and the lowest index that has it.
__device__ __forceinline__ void wave_best(uint64_t& key, int& idx) {
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
        const uint64_t k = shfl_xor64(key, s);
        const int i = __shfl_xor(idx, s);
        if (k > key || (k == key && i < idx)) {
            key = k;
            idx = i;
        }
    }
}

template <int V, int TYPE>
__global__ __launch_bounds__(64 * kWaves) void gate_kernel(GateArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kWaves + threadIdx.x / 64;
    if (t >= a.T) return;
    double logit[V], score[V];
    uint64_t key[V];
    bool off[V];
    double top = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        float l = -INFINITY;
        if (e < a.E) {
            if constexpr (TYPE == MOE_F32)
                l = static_cast<const float*>(a.logits)[t * a.stride + e];
            else
                l = __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[t * a.stride + e] << 16);
        }
        logit[i] = (double)l;
        off[i] = l == -INFINITY;
        nan |= l != l;
        top = fmax(top, logit[i]);
    }
    if (a.score == MOE_SCORE_SOFTMAX) {
        top = __any(nan) ? NAN : wave_max(top);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            score[i] = off[i] ? 0.0 : exp(logit[i] - top);
            sum += score[i];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int i = 0; i < V; ++i) score[i] = off[i] ? (sum != sum ? sum : 0.0) : score[i] / sum;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) score[i] = 1.0 / (1.0 + exp(-logit[i]));
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        const double c = a.bias && e < a.E ? score[i] + (double)a.bias[e] : logit[i];
        off[i] |= c == -INFINITY;
        key[i] = off[i] ? 0 : order_key(c);
    }
    if (a.groups > 1) {
        // marks of all groups, lane g holding group g's (num_groups <= 64)
        const int n = a.E / a.groups;
        const bool pair = a.group_score == MOE_GROUP_TOP2;
        uint64_t mark = 0;
        for (int g = 0; g < a.groups; ++g) {
            uint64_t gk[2] = {0, 0};
            double gv[2] = {0.0, 0.0};
            int taken = -1;
            for (int r = 0; r < (pair ? 2 : 1); ++r) {
                uint64_t k = 0;
                int at = 1 << 30;
                double v = 0.0;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = lane + 64 * i;
                    if (e / n != g || e == taken || off[i]) continue;
                    const double c = a.bias ? score[i] + (double)a.bias[e] : pair ? score[i] : logit[i];
                    const uint64_t ck = order_key(c);
                    if (ck > k) {
                        k = ck;
                        at = e;
                        v = c;
                    }
                }
                const int mine = at;
                wave_best(k, at);
                if (k == 0) break;
                taken = at;
                gk[r] = k;
                gv[r] = wave_max(mine == at ? (v != v ? NAN : v) : -INFINITY);
                if (__any(mine == at && v != v)) gv[r] = NAN;
            }
            const uint64_t m = gk[0] == 0 ? 0 : pair && gk[1] != 0 ? order_key(gv[0] + gv[1]) : gk[0];
            if (lane == g) mark = m;
        }
        uint64_t held = 0;
        for (int r = 0; r < a.topk_groups; ++r) {
            uint64_t k = lane < a.groups && !((held >> lane) & 1) ? mark : 0;
            int at = lane;
            wave_best(k, at);
            if (k == 0) break;
            held |= 1ull << at;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 64 * i;
            if (e < a.E && !((held >> (e / n)) & 1)) key[i] = 0;
        }
    }
    // lane j keeps the j-th choice
    int my_id = -1;
    double my_w = 0.0;
    for (int j = 0; j < a.k; ++j) {
        uint64_t k = 0;
        int at = 1 << 30;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] > k) {
                k = key[i];
                at = lane + 64 * i;
            }
        wave_best(k, at);
        if (k == 0) break;
        double w = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 64 * i == at) {
                key[i] = 0;
                w = score[i];
            }
        w = __shfl(w, at & 63);
        if (lane == j) {
            my_id = at;
            my_w = w;
        }
    }
    if (a.renorm) {
        const double sum = wave_sum(my_w);
        my_w = sum == 0.0 ? 0.0 : my_w / sum;
    }
    if (lane < a.k) {
        a.topk_idx[t * a.k + lane] = my_id;
        a.topk_w[t * a.k + lane] = (float)(my_id < 0 ? 0.0 : my_w * (double)a.scale);
    }
}

template <int V>
hipError_t launch(const GateArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)(((int64_t)a.T + kWaves - 1) / kWaves));
    if (a.logits_type == MOE_F32)
        hipLaunchKernelGGL((gate_kernel<V, MOE_F32>), grid, dim3(64 * kWaves), 0, stream, a);
    else
        hipLaunchKernelGGL((gate_kernel<V, MOE_BF16>), grid, dim3(64 * kWaves), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gate(const GateArgs& a, hipStream_t stream) {
    if (a.E <= 64) return launch<1>(a, stream);
    if (a.E <= 256) return launch<4>(a, stream);
    if (a.E <= 512) return launch<8>(a, stream);
    return launch<16>(a, stream);
}

}  // namespace moe
