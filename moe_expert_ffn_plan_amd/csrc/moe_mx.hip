// Microscaled quantisation: 32 neighbouring columns share a power-of-two scale 2^s, the smallest one that brings the
// block's largest magnitude to the format's largest value (6 in E2M1, 448 in E4M3) or below; codes are x / 2^s rounded
// to the nearest value of the format, ties to the even code.  The division is exact, so a code is one rounding of x.
#include "moe_internal.h"

namespace moe {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// 8 consecutive elements as they lie in memory.
template <int TYPE>
struct Raw;
template <>
struct Raw<MOE_BF16> {
    v4i v;
    __device__ __forceinline__ void load(const void* base, int64_t i) {
        v = *reinterpret_cast<const v4i*>(static_cast<const uint16_t*>(base) + i);
    }
    __device__ __forceinline__ float at(int j) const {
        const uint32_t w = (uint32_t)v[j >> 1];
        return __uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16);
    }
};
template <>
struct Raw<MOE_F32> {
    v4f v[2];
    __device__ __forceinline__ void load(const void* base, int64_t i) {
        const v4f* p = reinterpret_cast<const v4f*>(static_cast<const float*>(base) + i);
        v[0] = p[0];
        v[1] = p[1];
    }
    __device__ __forceinline__ float at(int j) const { return v[j >> 2][j & 3]; }
};

// Maximum over each four neighbouring lanes (quad_perm moves, inside the quad) of magnitudes as bit patterns, which
// order the same way and put infinity and NaN on top.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));
    return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));
}

// UE8M0 code of the smallest power of two 2^s with amax / 2^s <= 6 = 1.5 * 2^2, or 448 = 1.75 * 2^8.  At most 253, so
// that 2^-s is a normal number.
template <int FMT>
__device__ __forceinline__ int scale_code(uint32_t bits) {
    constexpr int EXP = FMT == MOE_E2M1 ? 2 : 8;
    constexpr uint32_t MANT = FMT == MOE_E2M1 ? 0x400000u : 0x600000u;
    const int c = (int)(bits >> 23) - EXP + ((bits & 0x7FFFFFu) > MANT ? 1 : 0);
    return c < 0 ? 0 : c;
}

constexpr uint32_t kInfinity = 0x7F800000u;
constexpr int kNanScale = 255;

// 8 columns of a row from their values: element i of the row-major outputs (a multiple of 8).
template <int XT, int FMT>
__device__ __forceinline__ void quant8(const MxQuantArgs& a, int64_t i, const Raw<XT>& x) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x.at(j)) & 0x7FFFFFFFu);
    m = quad_max(m);
    const bool whole = m < kInfinity;
    const int code = whole ? scale_code<FMT>(m) : kNanScale;
    // a block that holds an infinity or a NaN has no codes: its scale is NaN
    const float inv = whole ? __uint_as_float((uint32_t)(254 - code) << 23) : 0.0f;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = whole ? x.at(j) * inv : 0.0f;
    uint32_t q[2] = {0, 0};
    if constexpr (FMT == MOE_E2M1) {
        q[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q[0], v[0], v[1], 1.0f, 0);
        q[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q[0], v[2], v[3], 1.0f, 1);
        q[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q[0], v[4], v[5], 1.0f, 2);
        q[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q[0], v[6], v[7], 1.0f, 3);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int r = 0;
            r = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], r, false);
            r = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], r, true);
            q[h] = (uint32_t)r;
        }
    }
    if (a.x_q) {
        if constexpr (FMT == MOE_E2M1) *reinterpret_cast<uint32_t*>(a.x_q + i / 2) = q[0];
        else *reinterpret_cast<uint2*>(a.x_q + i) = make_uint2(q[0], q[1]);
        if ((i & 31) == 0) a.x_sf[i / 32] = (uint8_t)code;
    }
    if (a.x_dq) {
        f32x2 d[4];
        if constexpr (FMT == MOE_E2M1) {
            d[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.0f, 0);
            d[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.0f, 1);
            d[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.0f, 2);
            d[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.0f, 3);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                d[2 * h] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[h], false);
                d[2 * h + 1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[h], true);
            }
        }
        v4i o;
#pragma unroll
        for (int p = 0; p < 4; ++p)
            o[p] = whole ? (int)pack_bf16(ldexpf(d[p][0], code - 127), ldexpf(d[p][1], code - 127)) : 0x7FC07FC0;
        *reinterpret_cast<v4i*>(a.x_dq + i) = o;
    }
}

// One pass, bound by memory: x is read once, codes, scales and BF16 values are written once (16384 x 7168 BF16 to E2M1,
// 297 MB: 58-62 us, 4.8-5.1 TB/s; 16384 rows of 2048 of 4096 columns to E4M3, 102 MB: 18.8 us, 5.4 TB/s; a copy 5.1).  A
// lane takes 8 neighbouring columns, 16 or 32 bytes of x in one or two loads, so a block of 32 is four lanes and its maximum
// two moves within them: no LDS, no barrier.  A workgroup covers `lanes` lanes of each of 256 / lanes rows, so that short
// rows fill it too; rows without gaps count as one long row, and so do all outputs.
constexpr int kThreads = 256;
template <int XT, int FMT>
__global__ __launch_bounds__(kThreads) void mx_quant_kernel(MxQuantArgs a, int lanes, int64_t chunks) {
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int64_t row = block / chunks * (kThreads / lanes) + threadIdx.x / lanes;
    const int64_t c = (block % chunks * lanes + (threadIdx.x & (lanes - 1))) * 8;
    if (row >= a.rows || c >= a.cols) return;  // whole blocks of 32: lanes is a multiple of 4
    Raw<XT> x;
    x.load(a.x, row * a.stride + c);
    quant8<XT, FMT>(a, row * a.cols + c, x);
}

template <int XT, int FMT>
hipError_t launch(MxQuantArgs a, hipStream_t stream) {
    if (a.stride == a.cols || a.rows == 1) {
        a.cols *= a.rows;
        a.rows = 1;
        a.stride = a.cols;
    }
    int lanes = kThreads;
    while (lanes > 4 && (int64_t)(lanes / 2) * 8 >= a.cols) lanes /= 2;
    const int64_t chunks = (a.cols + (int64_t)lanes * 8 - 1) / ((int64_t)lanes * 8);
    const int64_t groups = (a.rows + kThreads / lanes - 1) / (kThreads / lanes);
    hipLaunchKernelGGL((mx_quant_kernel<XT, FMT>), wide_grid(chunks * groups), dim3(kThreads), 0, stream, a, lanes, chunks);
    return hipGetLastError();
}

// ---- weights of the dense product

// A thread writes one 16-byte slot of codes; see moe_linear.hip for the layout.
__global__ __launch_bounds__(kThreads) void tile_codes_kernel(const uint8_t* w, int N, int K, int KT, int64_t slots,
                                                              uint8_t* out) {
    const int64_t s = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
    if (s >= slots) return;
    const int p = (int)(s & 127), c = p >> 2, chunk = (p & 3) ^ ((c >> 2) & 3);
    const int64_t blk = s >> 7;
    const int kt = (int)(blk % KT);
    const int64_t nb = blk / KT;
    const int64_t n = (nb >> 1) * 64 + 2 * c + (nb & 1);
    const int64_t k = (int64_t)kt * 128 + chunk * 32;
    v4i v = {0, 0, 0, 0};
    if (n < N && k < K) v = *reinterpret_cast<const v4i*>(w + (n * K + k) / 2);
    *reinterpret_cast<v4i*>(out + s * 16) = v;
}
__global__ __launch_bounds__(kThreads) void tile_scales_kernel(const uint8_t* sf, int N, int K, int KT, int64_t words,
                                                               uint32_t* out) {
    const int64_t s = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
    if (s >= words) return;
    const int c = (int)(s & 31);
    const int64_t blk = s >> 5;
    const int kt = (int)(blk % KT);
    const int64_t nb = blk / KT;
    const int64_t n = (nb >> 1) * 64 + 2 * c + (nb & 1);
    uint32_t v = 0;
    if (n < N)
        for (int b = 0; b < 4; ++b) {
            const int64_t k = (int64_t)kt * 4 + b;
            if (k * 32 < K) v |= (uint32_t)sf[n * (K / 32) + k] << (8 * b);
        }
    out[s] = v;
}

}  // namespace

hipError_t launch_mx_quant(const MxQuantArgs& a, int x_type, int format, hipStream_t stream) {
    if (x_type == MOE_BF16)
        return format == MOE_E2M1 ? launch<MOE_BF16, MOE_E2M1>(a, stream) : launch<MOE_BF16, MOE_E4M3>(a, stream);
    return format == MOE_E2M1 ? launch<MOE_F32, MOE_E2M1>(a, stream) : launch<MOE_F32, MOE_E4M3>(a, stream);
}

hipError_t launch_mx_linear_prepare(int N, int K, const uint8_t* w, const uint8_t* w_sf, uint8_t* w_tiled,
                                    hipStream_t stream) {
    const int KT = mx_steps(K);
    const int64_t blocks = mx_column_blocks(N) * KT, slots = blocks * 128, words = blocks * 32;
    hipLaunchKernelGGL(tile_codes_kernel, wide_grid((slots + kThreads - 1) / kThreads), dim3(kThreads), 0, stream, w, N,
                       K, KT, slots, w_tiled);
    hipLaunchKernelGGL(tile_scales_kernel, wide_grid((words + kThreads - 1) / kThreads), dim3(kThreads), 0, stream, w_sf,
                       N, K, KT, words, reinterpret_cast<uint32_t*>(w_tiled + slots * 16));
    return hipGetLastError();
}

}  // namespace moe
