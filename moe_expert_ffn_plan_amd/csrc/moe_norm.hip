// Residual addition, RMS norm and E4M3 / UE8M0 quantisation of one row per token:
//   h = x + residual, v = h / sqrt(mean(h^2) + eps) * weight,
//   residual_out = h, y = BF16(v), x_q / x_sf = v per 32 columns with the power-of-two scale that brings
//   the block's largest magnitude to 448 or below.
//
// HBM-bound: a row is read once and written once (BF16 throughout: 2 + 2 bytes in, 2 + 2 + 1 + 1/32 out
// per element; 16384 x 7168: 1.06 GB in 180 us, 5.9 TB/s, where a copy of 2 GiB reaches 4.9 TB/s; with FP32 residual and
// weight 282 us, 5.4 TB/s; 256 rows of 65536, read twice, 36.5 us).  A lane owns
// 8 consecutive columns at a time (16 bytes of BF16), so a block of 32 columns is four neighbouring lanes and
// its maximum two DPP steps; the row stays in registers between the sum and the outputs.  Loads with the
// non-temporal hint lost (2048 x 4096: 11.9 -> 16.9 us, the inputs then miss the memory-side cache).
//
// Roundings: h is one FP32 addition for the outputs; the mean is that of the whole h, added and squared in FP64 (it
// decides the scale of every element of the row, and |h| above 2^64 must not overflow); v is two FP32 products.  The
// scale compares max|v| with 448 * 2^s: where the FP32 maximum lies within 4 units in the last place of that border,
// more than v's four roundings can move it (h, 1 / rms, two products: 4 * 2^-24 of 1.75 are 3.5 units), the block's
// maximum is formed again in FP64.
#include "moe_internal.h"

namespace moe {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

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

// LATER: not read again before a whole layer has run, so past the caches.
template <int TYPE, bool LATER>
__device__ __forceinline__ void store8(void* base, int64_t i, const float (&f)[8]) {
    auto put = [](auto v, auto* p) {
        if constexpr (LATER) __builtin_nontemporal_store(v, p);
        else *p = v;
    };
    if constexpr (TYPE == MOE_BF16) {
        v4i o;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = (int)pack_bf16(f[2 * q], f[2 * q + 1]);
        put(o, reinterpret_cast<v4i*>(static_cast<uint16_t*>(base) + i));
    } else {
        v4f* p = reinterpret_cast<v4f*>(static_cast<float*>(base) + i);
        put(v4f{f[0], f[1], f[2], f[3]}, p);
        put(v4f{f[4], f[5], f[6], f[7]}, p + 1);
    }
}

// x and the residual of 8 columns, and their h.
template <int XT, int RT>
struct Cell {
    Raw<XT> x;
    Raw<RT> r;
    __device__ __forceinline__ void load(const NormArgs& a, int64_t row, int c) {
        x.load(a.x, row * a.x_stride + c);
        if (a.residual) r.load(a.residual, row * a.residual_stride + c);
    }
    __device__ __forceinline__ void sum(const NormArgs& a, float (&h)[8]) const {
        if (a.residual) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = x.at(j) + r.at(j);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = x.at(j);
        }
    }
    // sum + the squares of h, each h whole (the FP32 h is, where nothing was added)
    __device__ __forceinline__ double squares(const NormArgs& a, const float (&h)[8], double sum) const {
        if (a.residual) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const double d = (double)x.at(j) + (double)r.at(j);
                sum = fma(d, d, sum);
            }
            if (sum > 0x1p255) {  // an h that FP32 does not hold is infinite here too: 2^256 or more of the sum
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = fabsf(h[j]) == INFINITY ? INFINITY : sum;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fma((double)h[j], (double)h[j], sum);
        }
        return sum;
    }
};

// Maximum over each four neighbouring lanes (quad_perm moves, inside the quad) of non-negative floats as
// bit patterns, which order the same way and put NaN on top.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));
    return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));
}

// UE8M0 code of the smallest power of two 2^s with amax / 2^s <= 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_code(uint32_t bits) {
    const int c = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return c < 0 ? 0 : c;
}

constexpr uint32_t kBorderUlp = 4;
__device__ __forceinline__ bool near_border(uint32_t bits) {
    return (bits & 0x7FFFFFu) - (0x600000u - kBorderUlp) <= 2 * kBorderUlp;
}

// scale_code of the block's maximum formed in FP64, for a block near a border; reads the columns again
// (before residual_out, which may be the same memory, is written).  All four lanes of the block call it.
template <int XT, int RT, int WT>
__device__ __forceinline__ int exact_code(const NormArgs& a, int64_t row, int c, double rstd) {
    Raw<XT> x;
    Raw<RT> r;
    Raw<WT> w;
    x.load(a.x, row * a.x_stride + c);
    w.load(a.weight, c);
    if (a.residual) r.load(a.residual, row * a.residual_stride + c);
    double m = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        double h = (double)x.at(j);
        if (a.residual) h += (double)r.at(j);
        m = fmax(m, fabs(h * rstd * (double)w.at(j)));
    }
    m = fmax(m, __shfl_xor(m, 1));
    m = fmax(m, __shfl_xor(m, 2));
    const uint64_t bits = (uint64_t)__double_as_longlong(m);
    const int e = (int)(bits >> 52) - 1023;
    const int code = e + 127 - 8 + ((bits & 0xFFFFFFFFFFFFFull) > 0xC000000000000ull ? 1 : 0);
    return code < 0 ? 0 : code;
}

// Outputs of 8 columns from their h.
template <int XT, int RT, int WT>
__device__ __forceinline__ void finish8(const NormArgs& a, int64_t row, int c, const float (&h)[8], const Raw<WT>& w,
                                        double rstd) {
    // FP32 holds 1 / rms in full once h is brought near 1 by a power of two, where it is far from it (an rms of
    // subnormals has a 1 / rms beyond FP32's range, one near the largest value a subnormal 1 / rms).
    const float by = (float)rstd;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = h[j] * by * w.at(j);
    // An rms of subnormals has a 1 / rms beyond FP32's range, one near the largest value a subnormal 1 / rms: far from
    // 1, h is brought near it by a power of two first.
    if (__builtin_expect(!(by < 0x1p64f && by > 0x1p-64f), 0)) {
        const float up = by < 1.0f ? 0x1p-64f : 0x1p96f, rest = (float)(rstd * (by < 1.0f ? 0x1p64 : 0x1p-96));
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = h[j] * up * rest * w.at(j);
    }
    if (a.x_q) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        m = quad_max(m);
        int code = scale_code(m);
        if (near_border(m)) code = exact_code<XT, RT, WT>(a, row, c, rstd);
        const float inv = __uint_as_float((uint32_t)(254 - code) << 23);  // 2^(127 - code)
        int q0 = 0, q1 = 0;
        q0 = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, q0, false);
        q0 = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, q0, true);
        q1 = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * inv, v[5] * inv, q1, false);
        q1 = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * inv, v[7] * inv, q1, true);
        *reinterpret_cast<int2*>(a.x_q + row * a.H + c) = make_int2(q0, q1);
        if ((c & 31) == 0) a.x_sf[row * (a.H / 32) + c / 32] = (uint8_t)code;
    }
    if (a.residual_out) store8<RT, true>(a.residual_out, row * a.residual_out_stride + c, h);
    if (a.y) store8<MOE_BF16, false>(a.y, row * a.H + c, v);
}

template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xF, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
    return v + __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
// Sum over each L = 8, 16, 32 or 64 neighbouring lanes, in all of them: inside rows of 16 lanes by DPP, across
// rows and halves by swaps.
template <int L>
__device__ __forceinline__ double lanes_sum(double v) {
    v = add_dpp<0xB1>(v);   // lane ^ 1
    v = add_dpp<0x4E>(v);   // lane ^ 2
    v = add_dpp<0x141>(v);  // lane ^ 7
    if constexpr (L > 8) v = add_dpp<0x140>(v);  // lane ^ 15
#pragma unroll
    for (int half = 0; half < (L == 64 ? 2 : L == 32 ? 1 : 0); ++half) {
        const uint64_t b = (uint64_t)__double_as_longlong(v);
        const uint32_t lo = (uint32_t)b, hi = (uint32_t)(b >> 32);
        const auto l = half ? __builtin_amdgcn_permlane32_swap(lo, lo, false, false)
                            : __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
        const auto h = half ? __builtin_amdgcn_permlane32_swap(hi, hi, false, false)
                            : __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
        v = __longlong_as_double((long long)(((uint64_t)h[0] << 32) | l[0])) +
            __longlong_as_double((long long)(((uint64_t)h[1] << 32) | l[1]));
    }
    return v;
}
// Sum over the workgroup, in all threads; part: one double per wave.
__device__ __forceinline__ double group_sum(double v, double* part) {
    v = lanes_sum<64>(v);
    const int waves = blockDim.x / 64;
    if (waves == 1) return v;
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = v;
    __syncthreads();
    v = 0.0;
    for (int i = 0; i < waves; ++i) v += part[i];
    return v;
}

// Rows of up to 8 L columns, 64 / L of them in a wave.
constexpr int kShortThreads = 256;
template <int XT, int RT, int WT, int L>
__global__ __launch_bounds__(kShortThreads) void norm_short_kernel(NormArgs a) {
    const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (kShortThreads / L) + threadIdx.x / L;
    const int64_t row = min(t, (int64_t)a.T - 1);  // lanes past the last row repeat it, and store nothing
    const int c = (threadIdx.x & (L - 1)) * 8, at = min(c, a.H - 8);
    Cell<XT, RT> cell;
    Raw<WT> w;
    cell.load(a, row, at);
    w.load(a.weight, at);
    float h[8];
    cell.sum(a, h);
    const double sum = lanes_sum<L>(c < a.H ? cell.squares(a, h, 0.0) : 0.0);
    const double rstd = 1.0 / sqrt(sum / a.H + (double)a.eps);
    if (t < a.T && c < a.H) finish8<XT, RT, WT>(a, row, c, h, w, rstd);
}

constexpr int kMaxThreads = 1024;

// One workgroup per row, the row in registers: V cells of 8 columns per thread, the threads' first cells side
// by side.
template <int XT, int RT, int WT, int V>
__global__ __launch_bounds__(kMaxThreads) void norm_row_kernel(NormArgs a) {
    __shared__ double part[kMaxThreads / 64];
    const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (row >= a.T) return;
    const int step = blockDim.x * 8;
    Cell<XT, RT> cell[V];
#pragma unroll
    for (int i = 0; i < V; ++i) cell[i].load(a, row, min((int)threadIdx.x * 8 + i * step, a.H - 8));
    Raw<WT> w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) w[i].load(a.weight, min((int)threadIdx.x * 8 + i * step, a.H - 8));
    float h[V][8];
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        cell[i].sum(a, h[i]);
        if ((int)threadIdx.x * 8 + i * step < a.H) sum = cell[i].squares(a, h[i], sum);
    }
    sum = group_sum(sum, part);
    const double rstd = 1.0 / sqrt(sum / a.H + (double)a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x * 8 + i * step;
        if (c < a.H) finish8<XT, RT, WT>(a, row, c, h[i], w[i], rstd);
    }
}

// Rows that the registers of a workgroup do not hold: two passes over the row.
template <int XT, int RT, int WT>
__global__ __launch_bounds__(kMaxThreads) void norm_long_kernel(NormArgs a) {
    __shared__ double part[kMaxThreads / 64];
    const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (row >= a.T) return;
    double sum = 0.0;
    for (int c = threadIdx.x * 8; c < a.H; c += kMaxThreads * 8) {
        Cell<XT, RT> cell;
        float h[8];
        cell.load(a, row, c);
        cell.sum(a, h);
        sum = cell.squares(a, h, sum);
    }
    sum = group_sum(sum, part);
    const double rstd = 1.0 / sqrt(sum / a.H + (double)a.eps);
    for (int c = threadIdx.x * 8; c < a.H; c += kMaxThreads * 8) {
        Cell<XT, RT> cell;
        Raw<WT> w;
        float h[8];
        cell.load(a, row, c);
        w.load(a.weight, c);
        cell.sum(a, h);
        finish8<XT, RT, WT>(a, row, c, h, w, rstd);
    }
}

template <int XT, int RT, int WT, int V>
hipError_t launch_row(const NormArgs& a, hipStream_t stream) {
    const int threads = (a.H / 8 + V * 64 - 1) / (V * 64) * 64;
    hipLaunchKernelGGL((norm_row_kernel<XT, RT, WT, V>), wide_grid(a.T), dim3((unsigned)threads), 0, stream, a);
    return hipGetLastError();
}

template <int XT, int RT, int WT, int L>
hipError_t launch_short(const NormArgs& a, hipStream_t stream) {
    constexpr int ROWS = kShortThreads / L;
    const dim3 grid = wide_grid(((int64_t)a.T + ROWS - 1) / ROWS);
    hipLaunchKernelGGL((norm_short_kernel<XT, RT, WT, L>), grid, dim3(kShortThreads), 0, stream, a);
    return hipGetLastError();
}

template <int XT, int RT, int WT>
hipError_t launch(const NormArgs& a, hipStream_t stream) {
    // Rows that leave half of a wave without work share it (65536 x 64: 7.2 us, 22.7 with a workgroup each; 65536 x
    // 256: 27.4, 29.6).
    if (a.H <= 64) return launch_short<XT, RT, WT, 8>(a, stream);
    if (a.H <= 128) return launch_short<XT, RT, WT, 16>(a, stream);
    if (a.H <= 256) return launch_short<XT, RT, WT, 32>(a, stream);
    // One cell per thread where rows are few (128 x 7168: 3.9 us against 4.1 with two and 4.7 with four) or
    // short (16384 x 1024: 28.8, 30.2, 29.5), else two: more loads in flight per thread, and at four too few
    // threads (16384 x 7168: 191, 180, 186).
    const int cells = a.H / 8;
    if (cells <= 256 || (a.T <= 256 && cells <= kMaxThreads)) return launch_row<XT, RT, WT, 1>(a, stream);
    if (cells <= 2 * kMaxThreads) return launch_row<XT, RT, WT, 2>(a, stream);
    if (cells <= 4 * kMaxThreads) return launch_row<XT, RT, WT, 4>(a, stream);
    hipLaunchKernelGGL((norm_long_kernel<XT, RT, WT>), wide_grid(a.T), dim3(kMaxThreads), 0, stream, a);
    return hipGetLastError();
}

template <int XT, int RT>
hipError_t launch_w(const NormArgs& a, hipStream_t stream) {
    return a.weight_type == MOE_BF16 ? launch<XT, RT, MOE_BF16>(a, stream) : launch<XT, RT, MOE_F32>(a, stream);
}

template <int XT>
hipError_t launch_r(const NormArgs& a, hipStream_t stream) {
    return a.residual_type == MOE_BF16 ? launch_w<XT, MOE_BF16>(a, stream) : launch_w<XT, MOE_F32>(a, stream);
}

}  // namespace

hipError_t launch_norm_quant(const NormArgs& a, hipStream_t stream) {
    return a.x_type == MOE_BF16 ? launch_r<MOE_BF16>(a, stream) : launch_r<MOE_F32>(a, stream);
}

}  // namespace moe
