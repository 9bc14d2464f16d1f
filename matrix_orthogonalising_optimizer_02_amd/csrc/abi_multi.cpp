// C ABI of the calls over many tensors: AdamW with 32-bit or 8-bit states, the gradient
// norm with its clip factor, and scaling in place. Declared in include/muon_rocm.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <string>
#include <vector>

#include "../../include/muon_rocm.h"
#include "abi_internal.hpp"
#include "train.hpp"

#define MUON_API extern "C" __attribute__((visibility("default")))

namespace muon {
namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
// A launch has at most 2^32 - 1 threads: in blocks of 256, or one of 1024 for each gradient's norm.
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;
constexpr int64_t kMaxBlocks = kMaxThreads / 256, kMaxTensors = kMaxThreads / 1024;
static_assert(kMultiThreads == 256, "a step's blocks");
constexpr int32_t kPlanAdamw = 0x41444d57, kPlanGrads = 0x4e4f524d;

// Blocks of the gradient norm: runs of at least 16384 elements, and longer ones where the
// set would take more than this many (the last launch adds their sums with one block).
constexpr int64_t kGradBlockElems = 16384;
constexpr int64_t kGradBlocks = 8192;

int fail(int code, const std::string& what) { return set_last_error(code, what); }
std::string at(int i) { return " at index " + std::to_string(i); }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int check_list(const void* list, int32_t count) {
    if (count < 0) return fail(MUON_ERR_INVALID_ARG, "count < 0");
    if (count > 0 && !list) return fail(MUON_ERR_INVALID_ARG, "the list of tensors is NULL");
    if (count >= kMaxTensors) return fail(MUON_ERR_TOO_LARGE, "more tensors than a launch takes");
    return MUON_OK;
}

int check_numel(int64_t n, int i) {
    if (n < 0) return fail(MUON_ERR_INVALID_ARG, "negative numel" + at(i));
    if (n > kMaxElems) return fail(MUON_ERR_TOO_LARGE, "tensor above 2^40 elements" + at(i));
    return MUON_OK;
}

int check_buffer(void* device, size_t bytes, size_t need, std::vector<Range>& ranges) {
    if (need == 0) return MUON_OK;
    if (!device) return fail(MUON_ERR_WORKSPACE, "device buffer is NULL");
    if (bytes < need) return fail(MUON_ERR_WORKSPACE, "device buffer too small: need " + std::to_string(need) + " bytes");
    if (addr(device) & 255) return fail(MUON_ERR_ALIGN, "device buffer not 256-byte aligned");
    ranges.push_back({addr(device), addr(device) + need, true});
    return MUON_OK;
}

struct Sizes {
    int64_t blocks = 0, block_elems = 0;
    size_t map = 0, partial = 0, bytes = 0;  // offsets and total of the device buffer
};

int adamw_sizes(const adamw_tensor* t, int32_t count, Sizes* s) {
    int rc = check_list(t, count);
    if (rc) return rc;
    for (int i = 0; i < count; ++i) {
        if ((rc = check_numel(t[i].numel, i))) return rc;
        s->blocks += ceil_div(t[i].numel, kMultiBlockElems);
    }
    if (s->blocks > kMaxBlocks) return fail(MUON_ERR_TOO_LARGE, "more blocks than a launch takes");
    s->map = align256(size_t(count) * sizeof(MultiDesc));
    // descriptors, the blocks' tensors, and the scalars of a step with a counter on the device
    s->bytes = s->blocks ? s->map + align256(size_t(s->blocks) * 4) + align256(sizeof(MultiScalars)) : 0;
    return MUON_OK;
}

int grad_sizes(const grad_tensor* t, int32_t count, Sizes* s) {
    int rc = check_list(t, count);
    if (rc) return rc;
    int64_t total = 0;
    for (int i = 0; i < count; ++i) {
        if ((rc = check_numel(t[i].numel, i))) return rc;
        total += t[i].numel;
    }
    s->block_elems = std::max(kGradBlockElems, ceil_div(ceil_div(total, kGradBlocks), kGradBlockElems) * kGradBlockElems);
    for (int i = 0; i < count; ++i) s->blocks += ceil_div(t[i].numel, s->block_elems);
    if (s->blocks > kMaxBlocks) return fail(MUON_ERR_TOO_LARGE, "more blocks than a launch takes");
    s->map = align256(size_t(count) * sizeof(GradDesc));
    s->partial = s->map + align256(size_t(s->blocks) * 4);
    s->bytes = count ? s->partial + align256(size_t(s->blocks) * 8) : 0;
    return MUON_OK;
}

int check_plan(const tensor_plan* p, int32_t kind) {
    if (!p) return fail(MUON_ERR_INVALID_ARG, "plan is NULL");
    if (p->kind != kind || p->count < 0 || p->blocks < 0 || (p->bytes && !p->device))
        return fail(MUON_ERR_INVALID_ARG, "not a plan of this call");
    return MUON_OK;
}

// A table that a capture records is not written: steps outside the graph, or before its
// first replay, would follow whatever addresses the buffer holds.
int check_not_capturing(hipStream_t s) {
    hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
    const hipError_t e = hipStreamIsCapturing(s, &status);
    if (e != hipSuccess) return fail(MUON_ERR_HIP, std::string("hipStreamIsCapturing: ") + hipGetErrorString(e));
    if (status != hipStreamCaptureStatusNone)
        return fail(MUON_ERR_INVALID_ARG, "a plan cannot be captured into a graph: make it before the capture");
    return MUON_OK;
}

// A plan's tables by its counts alone: the block length of a gradient plan is in `reserved`
// as a multiple of kGradBlockElems.
GradArgs grad_args(const tensor_plan& p) {
    GradArgs a{};
    char* base = static_cast<char*>(p.device);
    const size_t map = align256(size_t(p.count) * sizeof(GradDesc));
    a.table = reinterpret_cast<const GradDesc*>(base);
    a.tensor_of_block = reinterpret_cast<const int32_t*>(base + map);
    a.partial = reinterpret_cast<double*>(base + map + align256(size_t(p.blocks) * 4));
    a.block_elems = int64_t(p.reserved) * kGradBlockElems;
    a.count = p.count;
    a.blocks = p.blocks;
    return a;
}

}  // namespace
}  // namespace muon

using namespace muon;

MUON_API int adamw_multi_plan_bytes(const adamw_tensor* tensors, int32_t count, size_t* bytes) {
    return guarded([&]() -> int {
        if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
        Sizes sz;
        const int rc = adamw_sizes(tensors, count, &sz);
        if (rc == MUON_OK) *bytes = sz.bytes;
        return rc;
    });
}

MUON_API int adamw_multi_plan(const adamw_tensor* tensors, int32_t count, void* device, size_t bytes, tensor_plan* plan,
                              void* stream) {
    return guarded([&]() -> int {
        if (!plan) return fail(MUON_ERR_INVALID_ARG, "plan is NULL");
        Sizes sz;
        int rc = adamw_sizes(tensors, count, &sz);
        if (rc) return rc;
        std::vector<Range> ranges;
        int bits = -1;  // of all tensors so far; 0 once they differ
        for (int i = 0; i < count; ++i) {
            const adamw_tensor& t = tensors[i];
            if (t.numel == 0) continue;
            if (t.state_bits != 8 && t.state_bits != 32) return fail(MUON_ERR_INVALID_ARG, "state_bits must be 8 or 32" + at(i));
            const bool small = t.state_bits == 8;
            bits = bits < 0 || bits == t.state_bits ? t.state_bits : 0;
            if (!t.w || !t.g || !t.m || !t.v || (small && (!t.m_scale || !t.v_scale)))
                return fail(MUON_ERR_INVALID_ARG, "NULL pointer" + at(i));
            if (t.g_dtype < MUON_DTYPE_F32 || t.g_dtype > MUON_DTYPE_F16) return fail(MUON_ERR_INVALID_ARG, "unknown g_dtype" + at(i));
            if (t.copy && t.copy_dtype != MUON_DTYPE_BF16 && t.copy_dtype != MUON_DTYPE_F16)
                return fail(MUON_ERR_INVALID_ARG, "copy_dtype must be a 16-bit type" + at(i));
            if (!std::isfinite(t.lr_scale) || !std::isfinite(t.wd_scale))
                return fail(MUON_ERR_INVALID_ARG, "lr_scale and wd_scale must be finite" + at(i));
            if ((addr(t.w) | addr(t.g) | addr(t.m) | addr(t.v) | addr(t.copy)) & 15)
                return fail(MUON_ERR_ALIGN, "tensor pointer not 16-byte aligned" + at(i));
            if (small && ((addr(t.m_scale) | addr(t.v_scale)) & 3))
                return fail(MUON_ERR_ALIGN, "scales not 4-byte aligned" + at(i));
            const auto add = [&](const void* p, int64_t n, bool write) {
                ranges.push_back({addr(p), addr(p) + uintptr_t(n), write});
            };
            const int64_t state = t.numel * (small ? 1 : 4), scales = ceil_div(t.numel, kQBlock) * 4;
            add(t.w, t.numel * 4, true);
            add(t.m, state, true);
            add(t.v, state, true);
            add(t.g, t.numel * elem_size(t.g_dtype), false);
            if (t.copy) add(t.copy, t.numel * 2, true);
            if (small) {
                add(t.m_scale, scales, true);
                add(t.v_scale, scales, true);
            }
        }
        if ((rc = check_buffer(device, bytes, sz.bytes, ranges)) || (rc = check_overlaps(ranges))) return rc;
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        if (sz.blocks && (rc = check_not_capturing(s))) return rc;
        tensor_plan p{};
        p.device = device;
        p.bytes = sz.bytes;
        p.kind = kPlanAdamw;
        p.count = count;
        p.blocks = int32_t(sz.blocks);
        p.reserved = bits;
        *plan = p;
        if (sz.blocks == 0) return MUON_OK;
        MultiDescArgs a{};
        a.table = static_cast<MultiDesc*>(device);
        int32_t block = 0;
        for (int i = 0; i < count; ++i) {
            const adamw_tensor& t = tensors[i];
            MultiDesc& d = a.d[a.n++];
            d = MultiDesc{};
            d.w = t.w;
            d.copy = t.copy;
            d.g = t.g;
            d.m = t.m;
            d.v = t.v;
            d.ms = t.m_scale;
            d.vs = t.v_scale;
            d.n = t.numel;
            d.blk_begin = block;
            d.index = i;
            d.lr_scale = t.lr_scale;
            d.wd_scale = t.wd_scale;
            d.g_type = int8_t(t.g_dtype);
            d.copy_type = int8_t(t.copy_dtype);
            d.bits = int8_t(t.state_bits);
            block += int32_t(ceil_div(t.numel, kMultiBlockElems));
            if (a.n == kMultiPerLaunch || i == count - 1) {
                rc = run_timed(MUON_KCLASS_TENSOR_PLAN, s, "adamw table", [&] { return launch_multi_table(a, s); });
                if (rc) {
                    plan->kind = 0;
                    return rc;
                }
                a.first += a.n;
                a.n = 0;
            }
        }
        int32_t* map = reinterpret_cast<int32_t*>(static_cast<char*>(device) + sz.map);
        rc = run_timed(MUON_KCLASS_TENSOR_PLAN, s, "adamw map",
                       [&] { return launch_multi_map(a.table, count, map, int(sz.blocks), s); });
        if (rc) plan->kind = 0;
        return rc;
    });
}

namespace muon {
namespace {

int check_step(const tensor_plan* plan, const adamw_hparams* hp, const float* grad_scale) {
    const int rc = check_plan(plan, kPlanAdamw);
    if (rc) return rc;
    if (!hp) return fail(MUON_ERR_INVALID_ARG, "hparams is NULL");
    if (!std::isfinite(hp->lr) || !std::isfinite(hp->weight_decay))
        return fail(MUON_ERR_INVALID_ARG, "lr and weight_decay must be finite");
    if (!(hp->beta1 >= 0.f && hp->beta1 < 1.f) || !(hp->beta2 >= 0.f && hp->beta2 < 1.f))
        return fail(MUON_ERR_INVALID_ARG, "beta1 and beta2 must be in [0, 1)");
    if (!(hp->eps >= FLT_MIN) || !std::isfinite(hp->eps))
        return fail(MUON_ERR_INVALID_ARG, "eps must be a finite, normal number > 0");
    if (addr(grad_scale) & 3) return fail(MUON_ERR_ALIGN, "grad_scale not 4-byte aligned");
    return MUON_OK;
}

MultiArgs step_args(const tensor_plan& p, const adamw_hparams& hp, const float* grad_scale) {
    MultiArgs a{};
    a.table = static_cast<const MultiDesc*>(p.device);
    a.tensor_of_block = reinterpret_cast<const int32_t*>(static_cast<const char*>(p.device) +
                                                         align256(size_t(p.count) * sizeof(MultiDesc)));
    a.blocks = p.blocks;
    a.bits = p.reserved;
    a.beta1 = hp.beta1;
    a.beta2 = hp.beta2;
    a.one_minus_beta1 = float(1.0 - double(hp.beta1));
    a.one_minus_beta2 = float(1.0 - double(hp.beta2));
    a.eps = hp.eps;
    a.grad_scale = grad_scale;
    return a;
}

uint32_t seed_key(uint64_t seed) { return mix32(mix32(uint32_t(seed)) + uint32_t(seed >> 32)); }

}  // namespace
}  // namespace muon

MUON_API int adamw_multi_step(const tensor_plan* plan, const adamw_hparams* hp, int64_t step, uint64_t seed,
                              const float* grad_scale, void* stream) {
    return guarded([&]() -> int {
        const int rc = check_step(plan, hp, grad_scale);
        if (rc) return rc;
        if (step < 0) return fail(MUON_ERR_INVALID_ARG, "step < 0");
        if (plan->blocks == 0) return MUON_OK;
        // bias corrections in double on the host (t = step + 1)
        const double t = double(step) + 1.0;
        MultiArgs a = step_args(*plan, *hp, grad_scale);
        a.host.lr_bc1 = float(double(hp->lr) / (1.0 - std::pow(double(hp->beta1), t)));
        a.host.inv_sqrt_bc2 = float(1.0 / std::sqrt(1.0 - std::pow(double(hp->beta2), t)));
        a.host.lr_wd = double(hp->lr) * double(hp->weight_decay);
        a.host.key = mix32(seed_key(seed) + uint32_t(step));
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        return run_timed(MUON_KCLASS_ADAMW_MULTI, s, "adamw multi", [&] { return launch_multi_step(a, s); });
    });
}

MUON_API int adamw_multi_step_device(const tensor_plan* plan, const adamw_hparams* hp, int64_t* counter, const float* lr,
                                     uint64_t seed, const float* grad_scale, void* stream) {
    return guarded([&]() -> int {
        int rc = check_step(plan, hp, grad_scale);
        if (rc) return rc;
        if (!counter) return fail(MUON_ERR_INVALID_ARG, "counter is NULL");
        if (addr(counter) & 7) return fail(MUON_ERR_ALIGN, "counter not 8-byte aligned");
        if (addr(lr) & 3) return fail(MUON_ERR_ALIGN, "lr not 4-byte aligned");
        if (plan->blocks == 0) return MUON_OK;
        MultiArgs a = step_args(*plan, *hp, grad_scale);
        char* end = static_cast<char*>(plan->device) + plan->bytes;
        MultiScalarArgs m{};
        m.out = reinterpret_cast<MultiScalars*>(end - align256(sizeof(MultiScalars)));
        m.counter = counter;
        m.lr = lr;
        m.lr_host = hp->lr;
        m.beta1 = hp->beta1;
        m.beta2 = hp->beta2;
        m.weight_decay = hp->weight_decay;
        m.seed_key = seed_key(seed);
        a.scalars = m.out;
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        rc = run_timed(MUON_KCLASS_TENSOR_PLAN, s, "adamw scalars", [&] { return launch_multi_scalars(m, s); });
        if (rc) return rc;
        return run_timed(MUON_KCLASS_ADAMW_MULTI, s, "adamw multi", [&] { return launch_multi_step(a, s); });
    });
}

MUON_API int grad_norm_plan_bytes(const grad_tensor* grads, int32_t count, size_t* bytes) {
    return guarded([&]() -> int {
        if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
        Sizes sz;
        const int rc = grad_sizes(grads, count, &sz);
        if (rc == MUON_OK) *bytes = sz.bytes;
        return rc;
    });
}

MUON_API int grad_norm_plan(const grad_tensor* grads, int32_t count, void* device, size_t bytes, tensor_plan* plan,
                            void* stream) {
    return guarded([&]() -> int {
        if (!plan) return fail(MUON_ERR_INVALID_ARG, "plan is NULL");
        Sizes sz;
        int rc = grad_sizes(grads, count, &sz);
        if (rc) return rc;
        std::vector<Range> ranges;
        for (int i = 0; i < count; ++i) {
            const grad_tensor& t = grads[i];
            if (t.numel == 0) continue;
            if (!t.g) return fail(MUON_ERR_INVALID_ARG, "NULL pointer" + at(i));
            if (t.dtype < MUON_DTYPE_F32 || t.dtype > MUON_DTYPE_F16) return fail(MUON_ERR_INVALID_ARG, "unknown dtype" + at(i));
            const int e = elem_size(t.dtype);
            if (addr(t.g) % e) return fail(MUON_ERR_ALIGN, "gradient not aligned to its element" + at(i));
            ranges.push_back({addr(t.g), addr(t.g) + uintptr_t(t.numel) * e, true});
        }
        if ((rc = check_buffer(device, bytes, sz.bytes, ranges)) || (rc = check_overlaps(ranges))) return rc;
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        if (count && (rc = check_not_capturing(s))) return rc;
        tensor_plan p{};
        p.device = device;
        p.bytes = sz.bytes;
        p.kind = kPlanGrads;
        p.count = count;
        p.blocks = int32_t(sz.blocks);
        p.reserved = int32_t(sz.block_elems / kGradBlockElems);
        *plan = p;
        if (count == 0) return MUON_OK;
        GradDescArgs a{};
        a.table = static_cast<GradDesc*>(device);
        int32_t block = 0;
        for (int i = 0; i < count; ++i) {
            GradDesc& d = a.d[a.n++];
            d = GradDesc{};
            d.g = grads[i].g;
            d.n = grads[i].numel;
            d.type = grads[i].dtype;
            d.blk_begin = block;
            block += int32_t(ceil_div(grads[i].numel, sz.block_elems));
            d.blk_end = block;
            if (a.n == kGradPerLaunch || i == count - 1) {
                rc = run_timed(MUON_KCLASS_TENSOR_PLAN, s, "gradient table", [&] { return launch_grad_table(a, s); });
                if (rc) {
                    plan->kind = 0;
                    return rc;
                }
                a.first += a.n;
                a.n = 0;
            }
        }
        if (sz.blocks == 0) return MUON_OK;
        int32_t* map = reinterpret_cast<int32_t*>(static_cast<char*>(device) + sz.map);
        rc = run_timed(MUON_KCLASS_TENSOR_PLAN, s, "gradient map",
                       [&] { return launch_grad_map(a.table, count, map, int(sz.blocks), s); });
        if (rc) plan->kind = 0;
        return rc;
    });
}

MUON_API int grad_norm(const tensor_plan* plan, float max_norm, float* total, float* norms, void* stream) {
    return guarded([&]() -> int {
        int rc = check_plan(plan, kPlanGrads);
        if (rc) return rc;
        if (!total) return fail(MUON_ERR_INVALID_ARG, "total is NULL");
        if (!(max_norm > 0.f) || !std::isfinite(max_norm)) return fail(MUON_ERR_INVALID_ARG, "max_norm must be finite and > 0");
        if ((addr(total) | addr(norms)) & 3) return fail(MUON_ERR_ALIGN, "total or norms not 4-byte aligned");
        std::vector<Range> ranges{{addr(total), addr(total) + 8, true},
                                  {addr(plan->device), addr(plan->device) + plan->bytes, true}};
        if (norms) ranges.push_back({addr(norms), addr(norms) + uintptr_t(plan->count) * 4, true});
        if ((rc = check_overlaps(ranges))) return rc;
        GradArgs a = grad_args(*plan);
        a.max_norm = max_norm;
        a.total = total;
        a.norms = norms;
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        if (a.blocks) {
            rc = run_timed(MUON_KCLASS_GRAD_NORM, s, "gradient norm", [&] { return launch_grad_norm(a, s); });
            if (rc) return rc;
        }
        return run_timed(MUON_KCLASS_GRAD_TOTAL, s, "gradient total", [&] { return launch_grad_total(a, s); });
    });
}

MUON_API int grad_scale(const tensor_plan* plan, const float* factor, void* stream) {
    return guarded([&]() -> int {
        const int rc = check_plan(plan, kPlanGrads);
        if (rc) return rc;
        if (!factor) return fail(MUON_ERR_INVALID_ARG, "factor is NULL");
        if (addr(factor) & 3) return fail(MUON_ERR_ALIGN, "factor not 4-byte aligned");
        GradArgs a = grad_args(*plan);
        a.factor = factor;
        if (a.blocks == 0) return MUON_OK;
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        return run_timed(MUON_KCLASS_GRAD_SCALE, s, "gradient scale", [&] { return launch_grad_scale(a, s); });
    });
}
