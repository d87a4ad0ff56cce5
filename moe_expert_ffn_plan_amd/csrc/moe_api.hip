// C ABI of the fused MoE expert FFN library: host-side validation,
// workspace carving and the kernel sequence
//   routing -> Linear1 (+SwiGLU/requant) -> Linear2 (+BF16) -> combine,
// all enqueued on the caller's stream.  Interface modelled on the pages'
// host API: a size query plus caller-owned buffer (SymmBuffer page,
// sections 5-6), one forward entry point with strict shape checks that
// answer "unsupported" (reading notes, "host-side checks").
#include <atomic>
#include <cfloat>
#include <cstring>
#include <mutex>

#include "moe_internal.h"

using namespace moe;

namespace {

constexpr int kMaxDevices = 64;
// 0 = unknown, 1 = gfx950, 2 = other architecture
std::atomic<int> g_arch_cache[kMaxDevices];

int check_arch_current() {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return MOE_ERR_HIP;
    return moe_device_supported(dev);
}

int check_shape(const moe_shape* s) {
    if (!s) return MOE_ERR_NULL;
    if (s->num_tokens < 0 || s->hidden <= 0 || s->intermediate <= 0) return MOE_ERR_SHAPE;
    if (s->num_experts < 1 || s->num_experts > kMaxExperts) return MOE_ERR_SHAPE;
    if (s->topk < 1 || s->topk > kMaxTopk) return MOE_ERR_SHAPE;
    if (!block_m_supported(s->block_m)) return MOE_ERR_SHAPE;
    if ((int64_t)s->num_tokens * s->topk >= (1ll << 30)) return MOE_ERR_SHAPE;
    if (!(s->swiglu_limit >= 0.0f && s->swiglu_limit <= 3.0e38f)) return MOE_ERR_SHAPE;  // also rejects NaN
    if (s->exact_silu != 0 && s->exact_silu != 1) return MOE_ERR_SHAPE;
    if (s->weight_layout != MOE_WEIGHTS_PLAIN && s->weight_layout != MOE_WEIGHTS_TILED) return MOE_ERR_SHAPE;
    if (s->hidden > (1 << 20) || s->intermediate > (1 << 20)) return MOE_ERR_SHAPE;
    if (s->hidden % 256 != 0 || s->intermediate % 128 != 0) return MOE_ERR_ALIGN;
    // kernels address each operand's rows with 32-bit offsets
    const int64_t lim = 1ll << 31;
    if ((int64_t)s->num_tokens * s->hidden >= lim) return MOE_ERR_SHAPE;
    if (capacity_rows(*s) * s->intermediate >= lim) return MOE_ERR_SHAPE;
    if ((int64_t)s->hidden * s->intermediate >= lim) return MOE_ERR_SHAPE;
    return MOE_OK;
}

// The calls that read weights: a valid shape that also declares the tiled layout.
int check_weight_shape(const moe_shape* s) {
    const int st = check_shape(s);
    if (st != MOE_OK) return st;
    return s->weight_layout == MOE_WEIGHTS_TILED ? MOE_OK : MOE_ERR_LAYOUT;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

extern "C" {

int moe_device_supported(int device) {
    if (device < 0) return MOE_ERR_HIP;
    if (device < kMaxDevices) {
        const int c = g_arch_cache[device].load(std::memory_order_relaxed);
        if (c == 1) return MOE_OK;
        if (c == 2) return MOE_ERR_ARCH;
    }
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, device) != hipSuccess) return MOE_ERR_HIP;
    const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (device < kMaxDevices) g_arch_cache[device].store(ok ? 1 : 2, std::memory_order_relaxed);
    return ok ? MOE_OK : MOE_ERR_ARCH;
}

const char* moe_status_str(int status) {
    switch (status) {
        case MOE_OK: return "ok";
        case MOE_ERR_NULL: return "null pointer";
        case MOE_ERR_SHAPE: return "unsupported shape";
        case MOE_ERR_ALIGN: return "misaligned pointer or dimension";
        case MOE_ERR_WORKSPACE: return "workspace too small";
        case MOE_ERR_ARCH: return "device is not gfx950";
        case MOE_ERR_HIP: return "HIP runtime error";
        case MOE_ERR_LAYOUT: return "weights not declared in the tiled layout";
        default: return "unknown status";
    }
}

int moe_capacity_rows(const moe_shape* shape, int64_t* rows) {
    if (!rows) return MOE_ERR_NULL;
    const int st = check_shape(shape);
    if (st != MOE_OK) return st;
    *rows = capacity_rows(*shape);
    return MOE_OK;
}

int moe_suggest_block_m(int64_t num_tokens, int32_t topk, int32_t num_experts, int32_t* block_m) {
    if (!block_m) return MOE_ERR_NULL;
    if (num_tokens < 0 || num_tokens >= (1ll << 40) || topk < 1 || topk > kMaxTopk || num_experts < 1)
        return MOE_ERR_SHAPE;
    // target rows = imbalance factor 2 x expected rows per expert (T * k / E); the smallest routing
    // block of the pages' ladder that holds the target, compared exactly in integers: 2 T k <= c E
    const int64_t twice_hits = 2 * num_tokens * topk;
    int32_t pick = kBlockLadder[kBlockLadderSize - 1];
    for (const int32_t c : kBlockLadder)
        if (twice_hits <= (int64_t)c * num_experts) {
            pick = c;
            break;
        }
    *block_m = pick;
    return MOE_OK;
}

int moe_gemm_launches(const moe_shape* shape, int32_t* expert_ffn, int32_t* forward) {
    if (!expert_ffn || !forward) return MOE_ERR_NULL;
    const int st = check_shape(shape);
    if (st != MOE_OK) return st;
    *expert_ffn = fused_supported(*shape) ? 1 : 2;
    *forward = forward_one_launch(*shape, cu_count()) ? 1 : 2;
    return MOE_OK;
}

int moe_plan_workspace_bytes(const moe_shape* shape, size_t* bytes) {
    if (!bytes) return MOE_ERR_NULL;
    const int st = check_shape(shape);
    if (st != MOE_OK) return st;
    *bytes = plan_layout(*shape).total;
    return MOE_OK;
}

int moe_forward_workspace_bytes(const moe_shape* shape, size_t* bytes) {
    if (!bytes) return MOE_ERR_NULL;
    const int st = check_shape(shape);
    if (st != MOE_OK) return st;
    *bytes = forward_layout(*shape).total;
    return MOE_OK;
}

int moe_plan_view_get(const moe_shape* shape, void* plan_ws, moe_plan_view* out) {
    if (!out || !plan_ws) return MOE_ERR_NULL;
    const int st = check_shape(shape);
    if (st != MOE_OK) return st;
    const PlanLayout L = plan_layout(*shape);
    const PlanPtrs p = plan_ptrs(L, plan_ws);
    out->scalars = p.scalars; out->counts = p.counts; out->offsets = p.offsets; out->slot = p.slot;
    out->row_token = p.row_token; out->row_topk = p.row_topk; out->block_expert = p.block_expert;
    out->slack = p.slack; out->pull_order = p.pull_order; out->capacity_rows = L.cap;
    return MOE_OK;
}

int moe_forward_view_get(const moe_shape* shape, void* ws, moe_forward_view* out) {
    if (!out || !ws) return MOE_ERR_NULL;
    const int st = check_shape(shape);
    if (st != MOE_OK) return st;
    const ForwardLayout F = forward_layout(*shape);
    char* b = static_cast<char*>(ws);
    out->h_q = reinterpret_cast<uint8_t*>(b + F.h_q);
    out->h_sf = reinterpret_cast<uint8_t*>(b + F.h_sf);
    out->yslot = reinterpret_cast<uint16_t*>(b + F.yslot);
    out->plan = b + F.plan_base;
    out->capacity_rows = F.plan.cap;
    out->sync_status = reinterpret_cast<uint32_t*>(b + F.status);
    return MOE_OK;
}

int moe_plan(const moe_shape* shape, const int64_t* topk_idx, void* plan_ws, size_t plan_ws_bytes,
             void* stream) {
    int st = check_shape(shape);
    if (st != MOE_OK) return st;
    if (shape->num_tokens == 0) return MOE_OK;
    if (!topk_idx || !plan_ws) return MOE_ERR_NULL;
    if (!aligned(topk_idx, 8) || !aligned(plan_ws, kAlign)) return MOE_ERR_ALIGN;
    const PlanLayout L = plan_layout(*shape);
    if (plan_ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    if ((st = check_arch_current()) != MOE_OK) return st;
    const hipError_t e = launch_route(*shape, topk_idx, plan_ptrs(L, plan_ws), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int moe_prepare_weights(const moe_shape* shape, int which, const uint8_t* w, const uint8_t* w_sf, uint8_t* w_tiled,
                        uint8_t* w_sf_tiled, void* stream) {
    int st = check_shape(shape);
    if (st != MOE_OK) return st;
    if (which != 1 && which != 2) return MOE_ERR_SHAPE;
    if (!w || !w_sf || !w_tiled || !w_sf_tiled) return MOE_ERR_NULL;
    if (!aligned(w, 16) || !aligned(w_tiled, 16) || !aligned(w_sf, 4) || !aligned(w_sf_tiled, 4))
        return MOE_ERR_ALIGN;
    if ((st = check_arch_current()) != MOE_OK) return st;
    const int N = which == 1 ? 2 * shape->intermediate : shape->hidden;
    const int K = which == 1 ? shape->hidden : shape->intermediate;
    const hipError_t e = launch_tile_weights(which, N, K, shape->num_experts, w, w_sf, w_tiled, w_sf_tiled,
                                             static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int moe_linear1(const moe_shape* shape, const uint8_t* x, const uint8_t* x_sf, const float* topk_w,
                const uint8_t* w1, const uint8_t* w1_sf, const void* plan_ws, void* ws, size_t ws_bytes,
                void* stream) {
    int st = check_weight_shape(shape);
    if (st != MOE_OK) return st;
    if (shape->num_tokens == 0) return MOE_OK;
    if (!x || !x_sf || !topk_w || !w1 || !w1_sf || !plan_ws || !ws) return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(x_sf, 16) || !aligned(w1, 16) || !aligned(w1_sf, 16) || !aligned(topk_w, 4) ||
        !aligned(ws, kAlign) || !aligned(plan_ws, kAlign))
        return MOE_ERR_ALIGN;
    const ForwardLayout F = forward_layout(*shape);
    if (ws_bytes < F.total) return MOE_ERR_WORKSPACE;
    if ((st = check_arch_current()) != MOE_OK) return st;
    const PlanPtrs p = plan_ptrs(F.plan, const_cast<void*>(plan_ws));
    char* base = static_cast<char*>(ws);
    const GemmProblem g{shape, &p, F.plan.cap};
    const hipError_t e = launch_linear1(g, x, x_sf, topk_w, w1, w1_sf, reinterpret_cast<uint8_t*>(base + F.h_q),
                                        reinterpret_cast<uint8_t*>(base + F.h_sf),
                                        reinterpret_cast<uint32_t*>(base + F.status), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int moe_linear2(const moe_shape* shape, const uint8_t* w2, const uint8_t* w2_sf, const void* plan_ws, void* ws,
                size_t ws_bytes, void* stream) {
    int st = check_weight_shape(shape);
    if (st != MOE_OK) return st;
    if (shape->num_tokens == 0) return MOE_OK;
    if (!w2 || !w2_sf || !plan_ws || !ws) return MOE_ERR_NULL;
    if (!aligned(w2, 16) || !aligned(w2_sf, 16) || !aligned(ws, kAlign) || !aligned(plan_ws, kAlign))
        return MOE_ERR_ALIGN;
    const ForwardLayout F = forward_layout(*shape);
    if (ws_bytes < F.total) return MOE_ERR_WORKSPACE;
    if ((st = check_arch_current()) != MOE_OK) return st;
    const PlanPtrs p = plan_ptrs(F.plan, const_cast<void*>(plan_ws));
    char* base = static_cast<char*>(ws);
    const GemmProblem g{shape, &p, F.plan.cap};
    const hipError_t e = launch_linear2(g, reinterpret_cast<uint8_t*>(base + F.h_q),
                                        reinterpret_cast<uint8_t*>(base + F.h_sf), w2, w2_sf,
                                        reinterpret_cast<uint16_t*>(base + F.yslot), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"

namespace {
// moe_expert_ffn; prepared: the routing kernels enqueued just before did the single launch's prepare
// work (moe_forward building its plan inside ws), so no prepare kernel is enqueued.
int expert_ffn_call(const moe_shape* shape, const uint8_t* x, const uint8_t* x_sf, const float* topk_w,
                    const uint8_t* w1, const uint8_t* w1_sf, const uint8_t* w2, const uint8_t* w2_sf,
                    const void* plan_ws, void* ws, size_t ws_bytes, void* stream, bool prepared) {
    int st = check_weight_shape(shape);
    if (st != MOE_OK) return st;
    if (shape->num_tokens == 0) return MOE_OK;
    if (!x || !x_sf || !topk_w || !w1 || !w1_sf || !w2 || !w2_sf || !plan_ws || !ws) return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(x_sf, 16) || !aligned(w1, 16) || !aligned(w1_sf, 16) || !aligned(w2, 16) ||
        !aligned(w2_sf, 16) || !aligned(topk_w, 4) || !aligned(ws, kAlign) || !aligned(plan_ws, kAlign))
        return MOE_ERR_ALIGN;
    const ForwardLayout F = forward_layout(*shape);
    if (ws_bytes < F.total) return MOE_ERR_WORKSPACE;
    if ((st = check_arch_current()) != MOE_OK) return st;
    const PlanPtrs p = plan_ptrs(F.plan, const_cast<void*>(plan_ws));
    char* base = static_cast<char*>(ws);
    const GemmProblem g{shape, &p, F.plan.cap};
    const hipError_t e = launch_expert_ffn(
        g, x, x_sf, topk_w, w1, w1_sf, reinterpret_cast<uint8_t*>(base + F.h_q),
        reinterpret_cast<uint8_t*>(base + F.h_sf), w2, w2_sf, reinterpret_cast<uint16_t*>(base + F.yslot),
        reinterpret_cast<uint32_t*>(base + F.flags), reinterpret_cast<uint32_t*>(base + F.status),
        reinterpret_cast<uint32_t*>(base + F.epoch), static_cast<hipStream_t>(stream), prepared);
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
}  // namespace

extern "C" {

int moe_expert_ffn(const moe_shape* shape, const uint8_t* x, const uint8_t* x_sf, const float* topk_w,
                   const uint8_t* w1, const uint8_t* w1_sf, const uint8_t* w2, const uint8_t* w2_sf,
                   const void* plan_ws, void* ws, size_t ws_bytes, void* stream) {
    return expert_ffn_call(shape, x, x_sf, topk_w, w1, w1_sf, w2, w2_sf, plan_ws, ws, ws_bytes, stream, false);
}

int moe_combine(const moe_shape* shape, const void* plan_ws, const void* ws, size_t ws_bytes, uint16_t* y,
                void* stream) {
    int st = check_shape(shape);
    if (st != MOE_OK) return st;
    if (shape->num_tokens == 0) return MOE_OK;
    if (!plan_ws || !ws || !y) return MOE_ERR_NULL;
    if (!aligned(y, 16) || !aligned(ws, kAlign) || !aligned(plan_ws, kAlign)) return MOE_ERR_ALIGN;
    const ForwardLayout F = forward_layout(*shape);
    if (ws_bytes < F.total) return MOE_ERR_WORKSPACE;
    if ((st = check_arch_current()) != MOE_OK) return st;
    const PlanPtrs p = plan_ptrs(F.plan, const_cast<void*>(plan_ws));
    const char* base = static_cast<const char*>(ws);
    const hipError_t e = launch_combine(*shape, reinterpret_cast<const uint16_t*>(base + F.yslot), p.slot,
                                        reinterpret_cast<const uint32_t*>(base + F.status), y,
                                        static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int moe_forward(const moe_shape* shape, const uint8_t* x, const uint8_t* x_sf, const int64_t* topk_idx,
                const float* topk_w, const uint8_t* w1, const uint8_t* w1_sf, const uint8_t* w2,
                const uint8_t* w2_sf, uint16_t* y, const void* plan_ws, void* ws, size_t ws_bytes,
                void* stream) {
    int st = check_weight_shape(shape);
    if (st != MOE_OK) return st;
    if (shape->num_tokens == 0) return MOE_OK;
    if (!x || !x_sf || !topk_idx || !topk_w || !w1 || !w1_sf || !w2 || !w2_sf || !y || !ws) return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(x_sf, 16) || !aligned(w1, 16) || !aligned(w1_sf, 16) || !aligned(w2, 16) ||
        !aligned(w2_sf, 16) || !aligned(y, 16) || !aligned(topk_idx, 8) || !aligned(topk_w, 4) ||
        !aligned(ws, kAlign) || (plan_ws && !aligned(plan_ws, kAlign)))
        return MOE_ERR_ALIGN;
    const ForwardLayout F = forward_layout(*shape);
    if (ws_bytes < F.total) return MOE_ERR_WORKSPACE;
    if ((st = check_arch_current()) != MOE_OK) return st;
    char* base = static_cast<char*>(ws);
    const void* plan = plan_ws ? plan_ws : static_cast<const void*>(base + F.plan_base);
    const bool one_launch = forward_one_launch(*shape, cu_count());
    if (!plan_ws) {
        PlanPtrs pp = plan_ptrs(F.plan, base + F.plan_base);
        if (one_launch) {  // the routing kernels also do the single launch's prepare work
            pp.epoch_word = reinterpret_cast<uint32_t*>(base + F.epoch);
            pp.status = reinterpret_cast<uint32_t*>(base + F.status);
        }
        const hipError_t e = launch_route(*shape, topk_idx, pp, static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return MOE_ERR_HIP;
    }
    if (one_launch) {
        if ((st = expert_ffn_call(shape, x, x_sf, topk_w, w1, w1_sf, w2, w2_sf, plan, ws, ws_bytes, stream,
                                  !plan_ws)) != MOE_OK)
            return st;
    } else {
        if ((st = moe_linear1(shape, x, x_sf, topk_w, w1, w1_sf, plan, ws, ws_bytes, stream)) != MOE_OK) return st;
        if ((st = moe_linear2(shape, w2, w2_sf, plan, ws, ws_bytes, stream)) != MOE_OK) return st;
    }
    return moe_combine(shape, plan, ws, ws_bytes, y, stream);
}

// ---- allocation-free forward (moe_forward_noalloc)
// Its workspace is this file-scope device array: one copy per GPU, held until the process ends.  In
// host code the name `scratch` is only a host-side stand-in; the array's device address on a GPU comes
// from hipGetSymbolAddress, called once per device with that device current, and only that address is
// ever passed to kernels.
static __device__ __align__(256) uint8_t scratch[MOE_NOALLOC_WORKSPACE_BYTES];

}  // extern "C"

namespace {

std::mutex g_scratch_mu;
std::atomic<void*> g_scratch_ptr[kMaxDevices];

// Device address of `scratch` on the current device (resolved on the first call on that device).
int scratch_of_current_device(void** out) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return MOE_ERR_HIP;
    void* p = g_scratch_ptr[dev].load(std::memory_order_acquire);
    if (!p) {
        std::lock_guard<std::mutex> lock(g_scratch_mu);
        p = g_scratch_ptr[dev].load(std::memory_order_relaxed);
        if (!p) {
            if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return MOE_ERR_HIP;
            g_scratch_ptr[dev].store(p, std::memory_order_release);
        }
    }
    *out = p;
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_forward_noalloc(const moe_shape* shape, const uint8_t* x, const uint8_t* x_sf, const int64_t* topk_idx,
                        const float* topk_w, const uint8_t* w1, const uint8_t* w1_sf, const uint8_t* w2,
                        const uint8_t* w2_sf, uint16_t* y, void* stream) {
    int st = check_weight_shape(shape);
    if (st != MOE_OK) return st;
    if (shape->num_tokens == 0) return MOE_OK;
    if (!x || !x_sf || !topk_idx || !topk_w || !w1 || !w1_sf || !w2 || !w2_sf || !y) return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(x_sf, 16) || !aligned(w1, 16) || !aligned(w1_sf, 16) || !aligned(w2, 16) ||
        !aligned(w2_sf, 16) || !aligned(y, 16) || !aligned(topk_idx, 8) || !aligned(topk_w, 4))
        return MOE_ERR_ALIGN;
    if (forward_layout(*shape).total > (size_t)MOE_NOALLOC_WORKSPACE_BYTES) return MOE_ERR_WORKSPACE;
    if ((st = check_arch_current()) != MOE_OK) return st;
    void* ws = nullptr;
    if ((st = scratch_of_current_device(&ws)) != MOE_OK) return st;
    // the routing tables go to the plan region of the workspace (plan_ws = NULL)
    return moe_forward(shape, x, x_sf, topk_idx, topk_w, w1, w1_sf, w2, w2_sf, y, nullptr, ws,
                       (size_t)MOE_NOALLOC_WORKSPACE_BYTES, stream);
}

}  // extern "C"

// ---- in front of the experts
namespace {

bool type_ok(int t) { return t == MOE_BF16 || t == MOE_F32; }
bool flag_ok(int v) { return v == 0 || v == 1; }
bool tokens_ok(int t) { return t >= 0 && t < kMaxTokens; }  // tiles times threads fit a launch's 32 bits

// A stride as given (0 = contiguous) against the row length; vectors of 8 elements start every row.
int check_stride(int64_t stride, int64_t row) {
    if (stride == 0) return MOE_OK;
    if (stride < row || stride > (1ll << 40)) return MOE_ERR_SHAPE;
    return stride % 8 == 0 ? MOE_OK : MOE_ERR_ALIGN;
}
int64_t stride_or(int64_t stride, int64_t row) { return stride ? stride : row; }

int check_hidden(int h) {
    if (h <= 0 || h > kMaxHidden) return MOE_ERR_SHAPE;
    return h % 32 == 0 ? MOE_OK : MOE_ERR_ALIGN;
}

int check_norm(const moe_norm_shape* s) {
    if (!s) return MOE_ERR_NULL;
    if (!tokens_ok(s->num_tokens) || !type_ok(s->x_type) || !type_ok(s->residual_type) || !type_ok(s->weight_type))
        return MOE_ERR_SHAPE;
    if (!(s->eps >= 0.0f && s->eps <= FLT_MAX)) return MOE_ERR_SHAPE;  // also rejects NaN
    int st = check_hidden(s->hidden);
    for (const int64_t stride : {s->x_stride, s->residual_stride, s->residual_out_stride})
        if (st == MOE_OK) st = check_stride(stride, s->hidden);
    return st;
}

int check_router(const moe_router_shape* s) {
    if (!s) return MOE_ERR_NULL;
    if (!tokens_ok(s->num_tokens) || !type_ok(s->weight_type)) return MOE_ERR_SHAPE;
    if (s->num_experts < 1 || s->num_experts > kMaxGateExperts) return MOE_ERR_SHAPE;
    const int st = check_hidden(s->hidden);
    return st != MOE_OK ? st : check_stride(s->x_stride, s->hidden);
}

int check_gate(const moe_gate_shape* s) {
    if (!s) return MOE_ERR_NULL;
    if (!tokens_ok(s->num_tokens) || s->num_experts < 1 || s->num_experts > kMaxGateExperts) return MOE_ERR_SHAPE;
    if (s->num_groups < 1 || s->num_groups > kMaxGateGroups || s->num_experts % s->num_groups != 0)
        return MOE_ERR_SHAPE;
    if (s->topk_groups < 1 || s->topk_groups > s->num_groups) return MOE_ERR_SHAPE;
    if (s->topk < 1 || s->topk > kMaxTopk || s->topk > s->num_experts / s->num_groups * s->topk_groups)
        return MOE_ERR_SHAPE;
    if ((int64_t)s->num_tokens * s->topk >= (1ll << 30)) return MOE_ERR_SHAPE;
    if (!flag_ok(s->score) || !flag_ok(s->group_score) || !flag_ok(s->renormalize) || !type_ok(s->logits_type))
        return MOE_ERR_SHAPE;
    if (!(s->scale >= -FLT_MAX && s->scale <= FLT_MAX)) return MOE_ERR_SHAPE;  // also rejects NaN
    if (s->logits_stride != 0 && (s->logits_stride < s->num_experts || s->logits_stride > (1ll << 40)))
        return MOE_ERR_SHAPE;
    return MOE_OK;
}

GateArgs gate_args(const moe_gate_shape* s, const void* logits, const float* bias, int64_t* topk_idx, float* topk_w) {
    return GateArgs{logits, bias, topk_idx, topk_w, stride_or(s->logits_stride, s->num_experts), s->num_tokens,
                    s->num_experts, s->topk, s->num_groups, s->topk_groups, s->score, s->group_score, s->renormalize,
                    s->scale, s->logits_type};
}

}  // namespace

extern "C" {

int moe_norm_quant(const moe_norm_shape* shape, const void* x, const void* residual, const void* weight,
                   void* residual_out, uint16_t* y, uint8_t* x_q, uint8_t* x_sf, void* stream) {
    int st = check_norm(shape);
    if (st != MOE_OK) return st;
    if (shape->num_tokens == 0) return MOE_OK;
    if (!x || !weight || (!y && !x_q) || (x_q == nullptr) != (x_sf == nullptr)) return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(residual_out, 16) ||
        !aligned(y, 16) || !aligned(x_q, 16))
        return MOE_ERR_ALIGN;
    const int H = shape->hidden;
    const NormArgs a{x, residual, weight, residual_out, y, x_q, x_sf,
                     stride_or(shape->x_stride, H), stride_or(shape->residual_stride, H),
                     stride_or(shape->residual_out_stride, H), shape->num_tokens, H,
                     shape->x_type, shape->residual_type, shape->weight_type, shape->eps};
    // in place an output element lies where its own input was, or it overwrites another row's
    const bool rows = a.T > 1;
    if (residual_out && residual_out == residual && rows && a.residual_out_stride != a.residual_stride) return MOE_ERR_SHAPE;
    if (residual_out && residual_out == x &&
        ((rows && a.residual_out_stride != a.x_stride) || shape->residual_type != shape->x_type))
        return MOE_ERR_SHAPE;
    if ((st = check_arch_current()) != MOE_OK) return st;
    return launch_norm_quant(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int moe_router_weight_bytes(const moe_router_shape* shape, size_t* bytes) {
    if (!bytes) return MOE_ERR_NULL;
    const int st = check_router(shape);
    if (st != MOE_OK) return st;
    *bytes = (size_t)((shape->num_experts + 15) / 16) * 16 * shape->hidden * 2 * router_parts(shape->weight_type);
    return MOE_OK;
}

int moe_router_workspace_bytes(const moe_router_shape* shape, size_t* bytes) {
    if (!bytes) return MOE_ERR_NULL;
    const int st = check_router(shape);
    if (st != MOE_OK) return st;
    *bytes = choose_router(shape->num_tokens, shape->hidden, shape->num_experts, router_parts(shape->weight_type))
                 .workspace_bytes(shape->num_tokens, shape->num_experts);
    return MOE_OK;
}

int moe_router_max_workspace_bytes(const moe_router_shape* shape, size_t* bytes) {
    if (!bytes) return MOE_ERR_NULL;
    const int st = check_router(shape);
    if (st != MOE_OK) return st;
    *bytes = most_router_workspace(shape->num_tokens, shape->hidden, shape->num_experts, router_parts(shape->weight_type));
    return MOE_OK;
}

int moe_router_tile(const moe_router_shape* shape, int32_t* tokens, int32_t* experts, int32_t* splits) {
    if (!tokens || !experts || !splits) return MOE_ERR_NULL;
    const int st = check_router(shape);
    if (st != MOE_OK) return st;
    const RouterChoice c =
        choose_router(shape->num_tokens, shape->hidden, shape->num_experts, router_parts(shape->weight_type));
    *tokens = c.tokens;
    *experts = c.experts;
    *splits = c.splits;
    return MOE_OK;
}

int moe_router_prepare(const moe_router_shape* shape, const void* w, uint8_t* w_tiled, void* stream) {
    int st = check_router(shape);
    if (st != MOE_OK) return st;
    if (!w || !w_tiled) return MOE_ERR_NULL;
    if (!aligned(w, 16) || !aligned(w_tiled, 16)) return MOE_ERR_ALIGN;
    if ((st = check_arch_current()) != MOE_OK) return st;
    const hipError_t e = launch_router_prepare(shape->hidden, shape->num_experts, shape->weight_type, w, w_tiled,
                                               static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int moe_router_logits(const moe_router_shape* shape, const uint16_t* x, const uint8_t* w_tiled, float* logits,
                      void* ws, size_t ws_bytes, void* stream) {
    int st = check_router(shape);
    if (st != MOE_OK) return st;
    if (shape->num_tokens == 0) return MOE_OK;
    const int T = shape->num_tokens, H = shape->hidden, E = shape->num_experts;
    const int parts = router_parts(shape->weight_type);
    const RouterChoice choice = choose_router(T, H, E, parts);
    const size_t need = choice.workspace_bytes(T, E);
    if (!x || !w_tiled || !logits || (need > 0 && !ws)) return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(w_tiled, 16) || !aligned(logits, 16) || (need > 0 && !aligned(ws, kAlign)))
        return MOE_ERR_ALIGN;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE;
    if ((st = check_arch_current()) != MOE_OK) return st;
    const RouterArgs a{x, w_tiled, logits, static_cast<float*>(ws), stride_or(shape->x_stride, H), T, H, E, parts};
    return launch_router_logits(a, choice, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int moe_gate(const moe_gate_shape* shape, const void* logits, const float* bias, int64_t* topk_idx, float* topk_w,
             void* stream) {
    int st = check_gate(shape);
    if (st != MOE_OK) return st;
    if (shape->num_tokens == 0) return MOE_OK;
    if (!logits || !topk_idx || !topk_w) return MOE_ERR_NULL;
    if (!aligned(logits, shape->logits_type == MOE_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(topk_idx, 8) ||
        !aligned(topk_w, 4))
        return MOE_ERR_ALIGN;
    if ((st = check_arch_current()) != MOE_OK) return st;
    const GateArgs a = gate_args(shape, logits, bias, topk_idx, topk_w);
    return launch_gate(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int moe_gate_lanes(const moe_gate_shape* shape, int32_t* lanes, int32_t* values, int32_t* keys) {
    if (!lanes || !values || !keys) return MOE_ERR_NULL;
    const int st = check_gate(shape);
    if (st != MOE_OK) return st;
    const GateChoice c = choose_gate(gate_args(shape, nullptr, nullptr, nullptr, nullptr));
    *lanes = c.lanes;
    *values = c.values;
    *keys = c.list;
    return MOE_OK;
}

}  // extern "C"

// ---- microscaled quantisation and the dense product
namespace {

bool format_ok(int f) { return f == MOE_E2M1 || f == MOE_E4M3; }

int check_mx_quant(const moe_mx_quant_shape* s) {
    if (!s) return MOE_ERR_NULL;
    if (!tokens_ok(s->num_rows) || !type_ok(s->x_type) || !format_ok(s->format)) return MOE_ERR_SHAPE;
    const int st = check_hidden(s->num_cols);
    return st != MOE_OK ? st : check_stride(s->x_stride, s->num_cols);
}

int check_mx_linear(const moe_mx_linear_shape* s) {
    if (!s) return MOE_ERR_NULL;
    if (!tokens_ok(s->num_tokens) || !format_ok(s->x_format)) return MOE_ERR_SHAPE;
    if (s->out_features < 1 || s->out_features > kMaxHidden) return MOE_ERR_SHAPE;
    if (s->y_stride != 0 && (s->y_stride < s->out_features || s->y_stride > (1ll << 40))) return MOE_ERR_SHAPE;
    return check_hidden(s->in_features);
}

MxLinearChoice choice_of(const moe_mx_linear_shape* s) {
    return choose_mx_linear(s->num_tokens, s->out_features, s->in_features, s->x_format);
}

}  // namespace

extern "C" {

int moe_mx_quant(const moe_mx_quant_shape* shape, const void* x, uint8_t* x_q, uint8_t* x_sf, uint16_t* x_dq,
                 void* stream) {
    int st = check_mx_quant(shape);
    if (st != MOE_OK) return st;
    if (shape->num_rows == 0) return MOE_OK;
    if (!x || (!x_q && !x_dq) || (x_q == nullptr) != (x_sf == nullptr)) return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(x_q, 16) || !aligned(x_dq, 16)) return MOE_ERR_ALIGN;
    if ((st = check_arch_current()) != MOE_OK) return st;
    const MxQuantArgs a{x, x_q, x_sf, x_dq, shape->num_rows, shape->num_cols, stride_or(shape->x_stride, shape->num_cols)};
    const hipError_t e = launch_mx_quant(a, shape->x_type, shape->format, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int moe_mx_linear_weight_bytes(const moe_mx_linear_shape* shape, size_t* bytes) {
    if (!bytes) return MOE_ERR_NULL;
    const int st = check_mx_linear(shape);
    if (st != MOE_OK) return st;
    *bytes = (size_t)(mx_column_blocks(shape->out_features) * mx_steps(shape->in_features) * kMxBlockBytes);
    return MOE_OK;
}

int moe_mx_linear_prepare(const moe_mx_linear_shape* shape, const uint8_t* w, const uint8_t* w_sf, uint8_t* w_tiled,
                          void* stream) {
    int st = check_mx_linear(shape);
    if (st != MOE_OK) return st;
    if (!w || !w_sf || !w_tiled) return MOE_ERR_NULL;
    if (!aligned(w, 16) || !aligned(w_tiled, 16)) return MOE_ERR_ALIGN;
    if ((st = check_arch_current()) != MOE_OK) return st;
    const hipError_t e = launch_mx_linear_prepare(shape->out_features, shape->in_features, w, w_sf, w_tiled,
                                                  static_cast<hipStream_t>(stream));
    return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int moe_mx_linear_workspace_bytes(const moe_mx_linear_shape* shape, size_t* bytes) {
    if (!bytes) return MOE_ERR_NULL;
    const int st = check_mx_linear(shape);
    if (st != MOE_OK) return st;
    *bytes = shape->num_tokens ? choice_of(shape).workspace_bytes() : 0;
    return MOE_OK;
}

int moe_mx_linear_max_workspace_bytes(const moe_mx_linear_shape* shape, size_t* bytes) {
    if (!bytes) return MOE_ERR_NULL;
    const int st = check_mx_linear(shape);
    if (st != MOE_OK) return st;
    *bytes = most_mx_linear_workspace(shape->num_tokens, shape->out_features, shape->in_features, shape->x_format);
    return MOE_OK;
}

int moe_mx_linear_tile(const moe_mx_linear_shape* shape, int32_t* tokens, int32_t* outputs, int32_t* splits) {
    if (!tokens || !outputs || !splits) return MOE_ERR_NULL;
    const int st = check_mx_linear(shape);
    if (st != MOE_OK) return st;
    const MxLinearChoice c = choice_of(shape);
    *tokens = c.tokens;
    *outputs = c.columns;
    *splits = c.splits;
    return MOE_OK;
}

int moe_mx_linear(const moe_mx_linear_shape* shape, const uint8_t* x, const uint8_t* x_sf, const uint8_t* w_tiled,
                  uint16_t* y, void* ws, size_t ws_bytes, void* stream) {
    int st = check_mx_linear(shape);
    if (st != MOE_OK) return st;
    if (shape->num_tokens == 0) return MOE_OK;
    const MxLinearChoice choice = choice_of(shape);
    const size_t need = choice.workspace_bytes();
    if (!x || !x_sf || !w_tiled || !y || (need > 0 && !ws)) return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(x_sf, 4) || !aligned(w_tiled, 16) || !aligned(y, 4) ||
        (need > 0 && !aligned(ws, kAlign)))
        return MOE_ERR_ALIGN;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE;
    if ((st = check_arch_current()) != MOE_OK) return st;
    const MxLinearArgs a{x, x_sf, w_tiled, y, static_cast<uint8_t*>(ws), stride_or(shape->y_stride, shape->out_features),
                         shape->num_tokens, shape->out_features, shape->in_features, shape->x_format};
    return launch_mx_linear(a, choice, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"

// ---- balance of the load, and the gate's gradient
namespace {

constexpr int kMaxSeqs = 1 << 20;

int check_balance(const moe_balance_shape* s) {
    if (!s) return MOE_ERR_NULL;
    if (!tokens_ok(s->num_tokens) || s->num_experts < 1 || s->num_experts > kMaxGateExperts) return MOE_ERR_SHAPE;
    if (s->topk < 1 || s->topk > kMaxTopk || s->topk > s->num_experts) return MOE_ERR_SHAPE;
    if ((int64_t)s->num_tokens * s->topk >= (1ll << 30)) return MOE_ERR_SHAPE;
    if (s->num_seqs < 1 || s->num_seqs > kMaxSeqs || (int64_t)s->num_seqs * s->num_experts >= (1ll << 30))
        return MOE_ERR_SHAPE;
    if (!flag_ok(s->score) || !flag_ok(s->renormalize) || !type_ok(s->logits_type)) return MOE_ERR_SHAPE;
    if (!(s->scale >= -FLT_MAX && s->scale <= FLT_MAX)) return MOE_ERR_SHAPE;  // also rejects NaN
    if (s->logits_stride != 0 && (s->logits_stride < s->num_experts || s->logits_stride > (1ll << 40)))
        return MOE_ERR_SHAPE;
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_balance_workspace_bytes(const moe_balance_shape* shape, size_t* bytes) {
    if (!bytes) return MOE_ERR_NULL;
    const int st = check_balance(shape);
    if (st != MOE_OK) return st;
    *bytes = balance_workspace(shape->num_tokens, shape->num_experts, shape->num_seqs);
    return MOE_OK;
}

int moe_balance(const moe_balance_shape* shape, const void* logits, const int64_t* topk_idx, const int64_t* seq_offsets,
                int32_t* counts, int32_t* rows, float* share, float* loss, float* z, void* ws, size_t ws_bytes,
                void* stream) {
    int st = check_balance(shape);
    if (st != MOE_OK) return st;
    if (!seq_offsets && shape->num_seqs != 1) return MOE_ERR_SHAPE;
    if (z && shape->score != MOE_SCORE_SOFTMAX) return MOE_ERR_SHAPE;
    const bool scores = rows || share || loss || z;
    if (!counts && !scores) return MOE_ERR_NULL;
    if (!ws || (shape->num_tokens > 0 && (!topk_idx || (scores && !logits)))) return MOE_ERR_NULL;
    if (!aligned(logits, shape->logits_type == MOE_F32 ? 4 : 2) || !aligned(topk_idx, 8) || !aligned(seq_offsets, 8) ||
        !aligned(counts, 4) || !aligned(rows, 4) || !aligned(share, 4) || !aligned(loss, 4) || !aligned(z, 4) ||
        !aligned(ws, kAlign))
        return MOE_ERR_ALIGN;
    if (ws_bytes < balance_workspace(shape->num_tokens, shape->num_experts, shape->num_seqs)) return MOE_ERR_WORKSPACE;
    if ((st = check_arch_current()) != MOE_OK) return st;
    const BalanceArgs a{scores ? logits : nullptr, topk_idx, seq_offsets, stride_or(shape->logits_stride, shape->num_experts),
                        shape->num_tokens, shape->num_experts, shape->topk, shape->num_seqs, shape->score,
                        shape->logits_type, counts, rows, share, loss, z};
    return launch_balance(a, ws, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

int moe_gate_grad(const moe_balance_shape* shape, const void* logits, const int64_t* topk_idx,
                  const int64_t* seq_offsets, const int32_t* counts, const int32_t* rows, const float* d_loss,
                  const float* d_z, const float* d_topk_w, void* d_logits, void* stream) {
    int st = check_balance(shape);
    if (st != MOE_OK) return st;
    if (!seq_offsets && shape->num_seqs != 1) return MOE_ERR_SHAPE;
    if (d_z && shape->score != MOE_SCORE_SOFTMAX) return MOE_ERR_SHAPE;
    const int64_t stride = stride_or(shape->logits_stride, shape->num_experts);
    if (d_logits && d_logits == logits && shape->num_tokens > 1 && stride != shape->num_experts) return MOE_ERR_SHAPE;
    if (!d_loss && !d_z && !d_topk_w) return MOE_ERR_NULL;
    if (shape->num_tokens == 0) return MOE_OK;
    if (!logits || !d_logits || (d_topk_w && !topk_idx) || (d_loss && !counts) || ((d_loss || d_z) && !rows))
        return MOE_ERR_NULL;
    const int size = shape->logits_type == MOE_F32 ? 4 : 2;
    if (!aligned(logits, size) || !aligned(d_logits, size) || !aligned(topk_idx, 8) || !aligned(seq_offsets, 8) ||
        !aligned(counts, 4) || !aligned(rows, 4) || !aligned(d_loss, 4) || !aligned(d_z, 4) || !aligned(d_topk_w, 4))
        return MOE_ERR_ALIGN;
    if ((st = check_arch_current()) != MOE_OK) return st;
    const GateGradArgs a{logits, topk_idx, seq_offsets, counts, rows, d_loss, d_z, d_topk_w, d_logits, stride,
                         shape->num_tokens, shape->num_experts, shape->topk, shape->num_seqs, shape->score,
                         shape->renormalize, shape->logits_type, shape->scale};
    return launch_gate_grad(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
