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

// One wave per 16 tokens x 16 experts, operands straight from memory.
template <int P>
__global__ __launch_bounds__(64) void router_simple_kernel(RouterArgs a) {
    const int lane = threadIdx.x, KT = a.H / 32;
    const int t = blockIdx.y * 16 + (lane & 15);
    const uint16_t* x = a.x + (int64_t)min(t, a.T - 1) * a.x_stride + (lane >> 4) * 8;
    const uint8_t* w = a.w + ((int64_t)blockIdx.x * KT * P * 64 + lane) * 16;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    for (int kt = 0; kt < KT; ++kt) {
        const bf16x8 b = *reinterpret_cast<const bf16x8*>(x + kt * 32);
#pragma unroll
        for (int p = 0; p < P; ++p)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                *reinterpret_cast<const bf16x8*>(w + ((int64_t)kt * P + p) * 1024), b, acc, 0, 0, 0);
    }
    if (t < a.T) store_logits(a.logits, a.E, t, blockIdx.x * 16 + (lane >> 4) * 4, acc);
}

}  // namespace

size_t router_workspace_bytes(int, int, int, int) { return 0; }

hipError_t launch_router_prepare(int H, int E, int weight_type, const void* w, uint8_t* w_tiled, hipStream_t stream) {
    const int64_t slots = (int64_t)((E + 15) / 16) * (H / 32) * 64;
    const dim3 grid((unsigned)((slots + kThreads - 1) / kThreads));
    if (weight_type == MOE_F32)
        hipLaunchKernelGGL(router_prepare_kernel<MOE_F32>, grid, dim3(kThreads), 0, stream, w, H, E, slots, w_tiled);
    else
        hipLaunchKernelGGL(router_prepare_kernel<MOE_BF16>, grid, dim3(kThreads), 0, stream, w, H, E, slots, w_tiled);
    return hipGetLastError();
}

hipError_t launch_router_logits(const RouterArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.E + 15) / 16), (unsigned)((a.T + 15) / 16));
    if (a.parts == 3) hipLaunchKernelGGL(router_simple_kernel<3>, grid, dim3(64), 0, stream, a);
    else hipLaunchKernelGGL(router_simple_kernel<1>, grid, dim3(64), 0, stream, a);
    return hipGetLastError();
}

}  // namespace moe
