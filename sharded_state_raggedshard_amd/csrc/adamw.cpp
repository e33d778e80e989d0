// C-ABI entry points of AdamW over many tensors: the plan (work table), the
// tables of bound arrays, argument checks and launches.  Every check happens
// before the first launch.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <string>
#include <vector>

#include "adamw.hpp"
#include "raggedshard.h"
#include "row_checks.hpp"

struct rs_adamw {
    std::vector<rs_adamw_tensor> tensors;
    std::vector<rs::aw::Chunk> chunks;
    int64_t total = 0;      // elements of all tensors
    int32_t n_groups = 1;   // highest group + 1
    bool int8 = false;      // some tensor has 8-bit moments
    size_t off_chunks = 0, off_slots = 0, ws_bytes = 0;
    void* d_ws = nullptr;
    int device = -1;        // of the workspace
    bool uploaded = false, bound = false;
    // the bound arrays and the workspace by their first byte, and the furthest
    // end of the arrays up to each
    std::vector<uintptr_t> begin, end;
};

namespace {

using namespace rs::rowcheck;
using rs::aw::kChunk;

int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b != 0); }

int32_t block_log2(const rs_adamw_tensor& t) {
    int32_t l = 0;
    while ((int32_t(1) << l) < t.block) ++l;
    return l;
}

rs_status check_tensor(const rs_adamw_tensor& t) {
    if (t.numel < 0) return fail(RS_EINVAL, "negative number of elements");
    if (t.numel > rs::aw::kMaxElems) return fail(RS_EOVERFLOW, "a tensor beyond 2^42 elements");
    if ((t.param != RS_F32 && t.param != RS_BF16) || (t.grad != RS_F32 && t.grad != RS_BF16))
        return fail(RS_EINVAL, "unknown dtype");
    if (t.state != RS_STATE_F32 && t.state != RS_STATE_INT8 && t.state != RS_STATE_INT8_ROOT)
        return fail(RS_EINVAL, "unknown state");
    if (t.state == RS_STATE_F32 && t.block != 0) return fail(RS_EINVAL, "binary32 moments have no blocks");
    if (t.state != RS_STATE_F32 &&
        (t.block < (1 << rs::aw::kMinBlockLog2) || t.block > (1 << rs::aw::kMaxBlockLog2) ||
         (t.block & (t.block - 1)) != 0))
        return fail(RS_EINVAL, "block must be a power of two in 64..4096");
    if (t.group < 0 || t.group >= rs::aw::kMaxGroups) return fail(RS_EINVAL, "group outside 0..15");
    if (t.reserved != 0) return fail(RS_EINVAL, "reserved must be 0");
    return RS_OK;
}

rs::aw::Work work_of(const rs_adamw& h) {
    const char* w = static_cast<const char*>(h.d_ws);
    rs::aw::Work k;
    k.tensors = reinterpret_cast<const rs::aw::Tensor*>(w);
    k.chunks = reinterpret_cast<const rs::aw::Chunk*>(w + h.off_chunks);
    k.n_chunks = (int64_t)h.chunks.size();
    return k;
}

// A launch on another device than the workspace's could fault.
rs_status check_device(const rs_adamw* h) {
    int device = -1;
    hipError_t e = hipGetDevice(&device);
    if (e != hipSuccess) return hip_fail(e, "reading the current device");
    if (device != h->device) return fail(RS_ESTATE, "adamw plan uploaded on another device than the current one");
    return RS_OK;
}

rs_status check_ready(const rs_adamw* h) {
    if (!h->uploaded) return fail(RS_ESTATE, "adamw plan not uploaded");
    if (!h->bound) return fail(RS_ESTATE, "no tensors bound");
    return check_device(h);
}

// An array that a call writes beside the bound ones shares no byte with them.
rs_status check_free(const rs_adamw& h, const void* p, int64_t bytes) {
    if (!p || bytes == 0) return RS_OK;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = a + (uintptr_t)bytes;
    const size_t i = size_t(std::lower_bound(h.begin.begin(), h.begin.end(), b) - h.begin.begin());
    if (i > 0 && h.end[i - 1] > a) return fail(RS_EINVAL, "an output overlaps another array");
    return RS_OK;
}

// What is bound of one tensor, checked.
struct Span {
    uintptr_t a, b;
    bool written;
};

rs_status take(std::vector<Span>& spans, const void* p, int64_t bytes, size_t align, bool written) {
    if (bytes == 0) return RS_OK;
    if (!p) return fail(RS_EINVAL, "NULL argument");
    if (!aligned(p, align)) return fail(RS_EINVAL, "misaligned pointer");
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    spans.push_back({a, a + (uintptr_t)bytes, written});
    return RS_OK;
}

rs_status bind(rs_adamw* h, void* const* d_param, const void* const* d_grad, void* const* d_m,
               void* const* d_v, float* const* d_amax_m, float* const* d_amax_v,
               uint16_t* const* d_bf16_out, void* stream) {
    const size_t n = h->tensors.size();
    std::vector<rs::aw::Tensor> table(n);
    std::vector<Span> spans;
    spans.reserve(5 * n + 1);
    if (h->uploaded)
        spans.push_back({reinterpret_cast<uintptr_t>(h->d_ws), reinterpret_cast<uintptr_t>(h->d_ws) + h->ws_bytes, true});
    int64_t first = 0;
    for (size_t i = 0; i < n; ++i) {
        const rs_adamw_tensor& t = h->tensors[i];
        const bool eight = t.state != RS_STATE_F32;
        const int64_t psize = t.param == RS_F32 ? 4 : 2, gsize = t.grad == RS_F32 ? 4 : 2, ssize = eight ? 1 : 4;
        rs::aw::Tensor& d = table[i];
        d = rs::aw::Tensor{};
        d.param = d_param[i];
        d.grad = d_grad[i];
        d.m = d_m[i];
        d.v = d_v[i];
        d.out = d_bf16_out ? d_bf16_out[i] : nullptr;
        d.n = t.numel;
        d.first = first;
        d.kind = (t.param == RS_F32 ? rs::aw::KIND_PARAM_F32 : 0) | (t.grad == RS_F32 ? rs::aw::KIND_GRAD_F32 : 0) |
                 (eight ? rs::aw::KIND_INT8 : 0) | (t.state == RS_STATE_INT8_ROOT ? rs::aw::KIND_ROOT : 0);
        d.block_log2 = eight ? block_log2(t) : 0;
        d.group = t.group;
        first += t.numel;
        rs_status st = take(spans, d.param, t.numel * psize, size_t(psize), true);
        if (st == RS_OK) st = take(spans, d.grad, t.numel * gsize, size_t(gsize), false);
        if (st == RS_OK) st = take(spans, d.m, t.numel * ssize, size_t(ssize), true);
        if (st == RS_OK) st = take(spans, d.v, t.numel * ssize, size_t(ssize), true);
        if (st == RS_OK && eight) {
            d.amax_m = d_amax_m[i];
            d.amax_v = d_amax_v[i];
            const int64_t bytes = 4 * ceil_div(t.numel, t.block);
            st = take(spans, d.amax_m, bytes, 4, true);
            if (st == RS_OK) st = take(spans, d.amax_v, bytes, 4, true);
        }
        if (st == RS_OK && d.out && t.numel > 0) {
            if (t.param != RS_F32) return fail(RS_EINVAL, "a bf16 output beside bf16 parameters");
            st = take(spans, d.out, 2 * t.numel, 2, true);
        }
        if (st != RS_OK) return st;
    }
    // no written array shares a byte with another one
    std::sort(spans.begin(), spans.end(), [](const Span& x, const Span& y) { return x.a < y.a; });
    uintptr_t any = 0, written = 0;
    std::vector<uintptr_t> begin, end;
    begin.reserve(spans.size());
    end.reserve(spans.size());
    for (const Span& s : spans) {
        if (s.a < written || (s.written && s.a < any)) return fail(RS_EINVAL, "two of the arrays overlap");
        any = std::max(any, s.b);
        if (s.written) written = std::max(written, s.b);
        begin.push_back(s.a);
        end.push_back(any);
    }
    if (!h->uploaded) return fail(RS_ESTATE, "adamw plan not uploaded");
    rs_status at = check_device(h);
    if (at != RS_OK) return at;
    hipStream_t s = as_stream(stream);
    if (n > 0) {
        hipError_t e = hipMemcpyAsync(h->d_ws, table.data(), n * sizeof(rs::aw::Tensor), hipMemcpyHostToDevice, s);
        if (e == hipSuccess) e = hipStreamSynchronize(s);
        if (e != hipSuccess) {
            h->bound = false;
            return hip_fail(e, "copying the tensor table");
        }
    }
    h->begin.swap(begin);
    h->end.swap(end);
    h->bound = true;
    return RS_OK;
}

}  // namespace

extern "C" {

rs_status rs_adamw_plan(const rs_adamw_tensor* tensors, int32_t n, rs_adamw** out) {
    if (!out) return fail(RS_EINVAL, "NULL argument");
    *out = nullptr;
    if (n < 1 || !tensors) return fail(RS_EINVAL, "no tensors");
    int64_t chunks = 0, total = 0;
    for (int32_t i = 0; i < n; ++i) {
        rs_status st = check_tensor(tensors[i]);
        if (st != RS_OK) return st;
        chunks += ceil_div(tensors[i].numel, kChunk);
        total += tensors[i].numel;
        if (chunks > 0x7fffffff) return fail(RS_EOVERFLOW, "more than 2^31 - 1 chunks of work");
    }
    rs_adamw* h = nullptr;
    try {
        h = new rs_adamw;
        h->tensors.assign(tensors, tensors + n);
        h->chunks.reserve(size_t(chunks));
        for (int32_t i = 0; i < n; ++i) {
            for (int64_t c = 0; c < ceil_div(tensors[i].numel, kChunk); ++c) h->chunks.push_back({i, (int32_t)c});
            h->n_groups = std::max(h->n_groups, tensors[i].group + 1);
            h->int8 = h->int8 || tensors[i].state != RS_STATE_F32;
        }
    } catch (const std::bad_alloc&) {
        delete h;
        return fail(RS_ENOMEM, "host allocation failed");
    }
    h->total = total;
    h->off_chunks = align256(size_t(n) * sizeof(rs::aw::Tensor));
    h->off_slots = h->off_chunks + align256(h->chunks.size() * sizeof(rs::aw::Chunk));
    h->ws_bytes = h->off_slots + align256(rs::aw::kSumWords * sizeof(uint64_t));
    *out = h;
    return RS_OK;
}

void rs_adamw_free(rs_adamw* adamw) { delete adamw; }

size_t rs_adamw_device_bytes(const rs_adamw* adamw) {
    if (!adamw) {
        fail(RS_EINVAL, "adamw plan is NULL");
        return 0;
    }
    return adamw->ws_bytes;
}

rs_status rs_adamw_upload(rs_adamw* adamw, void* d_workspace, size_t bytes, void* stream) {
    if (!adamw) return fail(RS_EINVAL, "adamw plan is NULL");
    if (!d_workspace || !aligned(d_workspace, 256))
        return fail(RS_EINVAL, "workspace must be a non-NULL 256-byte aligned device pointer");
    if (bytes < adamw->ws_bytes) return fail(RS_ENOMEM, "workspace smaller than rs_adamw_device_bytes()");
    hipStream_t s = as_stream(stream);
    adamw->uploaded = adamw->bound = false;
    static const uint64_t zeros[rs::aw::kSumWords] = {};
    char* w = static_cast<char*>(d_workspace);
    hipError_t e = hipGetDevice(&adamw->device);
    if (e == hipSuccess) e = hipMemcpyAsync(w + adamw->off_slots, zeros, sizeof(zeros), hipMemcpyHostToDevice, s);
    if (e == hipSuccess && !adamw->chunks.empty())
        e = hipMemcpyAsync(w + adamw->off_chunks, adamw->chunks.data(), adamw->chunks.size() * sizeof(rs::aw::Chunk),
                           hipMemcpyHostToDevice, s);
    if (e == hipSuccess) e = hipStreamSynchronize(s);
    if (e != hipSuccess) return hip_fail(e, "copying the work table");
    adamw->d_ws = d_workspace;
    adamw->uploaded = true;
    return RS_OK;
}

rs_status rs_adamw_bind(rs_adamw* adamw, void* const* d_param, const void* const* d_grad, void* const* d_m,
                        void* const* d_v, float* const* d_amax_m, float* const* d_amax_v,
                        uint16_t* const* d_bf16_out, void* stream) {
    if (!adamw) return fail(RS_EINVAL, "adamw plan is NULL");
    if (!d_param || !d_grad || !d_m || !d_v || (adamw->int8 && (!d_amax_m || !d_amax_v)))
        return fail(RS_EINVAL, "NULL argument");
    try {
        return bind(adamw, d_param, d_grad, d_m, d_v, d_amax_m, d_amax_v, d_bf16_out, stream);
    } catch (const std::bad_alloc&) {
        return fail(RS_ENOMEM, "host allocation failed");
    }
}

rs_status rs_adamw_l2norm_clip(const rs_adamw* adamw, double max_norm, double* d_sumsq, float* d_scale, void* stream) {
    if (!adamw || !d_sumsq) return fail(RS_EINVAL, "NULL argument");
    if (!aligned(d_sumsq, 8) || !aligned(d_scale, 4)) return fail(RS_EINVAL, "misaligned pointer");
    if (d_scale && !(max_norm > 0.0 && std::isfinite(max_norm)))
        return fail(RS_EINVAL, "max_norm must be finite and > 0");
    rs_status st = check_apart({Extent{d_sumsq, 8}, Extent{d_scale, 4}}, {});
    if (st == RS_OK) st = check_ready(adamw);
    if (st == RS_OK) st = check_free(*adamw, d_sumsq, 8);
    if (st == RS_OK) st = check_free(*adamw, d_scale, 4);
    if (st != RS_OK) return st;
    uint64_t* slots = reinterpret_cast<uint64_t*>(static_cast<char*>(adamw->d_ws) + adamw->off_slots);
    hipError_t e = rs::aw::launch_l2norm(work_of(*adamw), slots, d_sumsq, max_norm, d_scale, as_stream(stream));
    if (e != hipSuccess) return hip_fail(e, "adamw norm launch");
    return RS_OK;
}

rs_status rs_adamw_step(const rs_adamw* adamw, const rs_adam_hparams* hp, int32_t n_groups,
                        const float* d_grad_scale, void* stream) {
    if (!adamw || !hp) return fail(RS_EINVAL, "NULL argument");
    if (n_groups < adamw->n_groups || n_groups > rs::aw::kMaxGroups)
        return fail(RS_EINVAL, "hyper-parameters for " + std::to_string(adamw->n_groups) + " to 16 groups needed");
    if (!aligned(d_grad_scale, 4)) return fail(RS_EINVAL, "misaligned pointer");
    rs::aw::Scalars sc{};
    for (int32_t i = 0; i < n_groups; ++i) {
        const rs_adam_hparams& p = hp[i];
        if (p.step < 1) return fail(RS_EINVAL, "step must be >= 1");
        if (!(p.beta1 >= 0.0 && p.beta1 < 1.0) || !(p.beta2 >= 0.0 && p.beta2 < 1.0) || !std::isfinite(p.lr) ||
            !std::isfinite(p.eps) || !std::isfinite(p.weight_decay))
            return fail(RS_EINVAL, "hyper-parameters out of range");
        // binary64 on the host, rounded once to binary32
        const double t = (double)p.step;
        rs::StepScalars& s = sc.group[i];
        s.beta1 = (float)p.beta1;
        s.beta2 = (float)p.beta2;
        s.omega1 = (float)(1.0 - p.beta1);
        s.omega2 = (float)(1.0 - p.beta2);
        s.eps = (float)p.eps;
        s.c_decay = (float)(1.0 - p.lr * p.weight_decay);
        s.step_size = (float)(p.lr / (1.0 - std::pow(p.beta1, t)));
        s.kappa = (float)(1.0 / std::sqrt(1.0 - std::pow(p.beta2, t)));
        s.limit = rs::update_limit(s.kappa, s.eps);
    }
    rs_status st = check_ready(adamw);
    if (st == RS_OK) st = check_free(*adamw, d_grad_scale, 4);
    if (st != RS_OK) return st;
    hipError_t e = rs::aw::launch_step(work_of(*adamw), sc, d_grad_scale, as_stream(stream));
    if (e != hipSuccess) return hip_fail(e, "adamw step launch");
    return RS_OK;
}

rs_status rs_adamw_moments(const rs_adamw* adamw, void* d_m, void* d_v, int32_t dtype, void* stream) {
    if (!adamw) return fail(RS_EINVAL, "NULL argument");
    if (dtype != RS_F32 && dtype != RS_BF16) return fail(RS_EINVAL, "unknown dtype");
    const int64_t size = dtype == RS_F32 ? 4 : 2;
    if (!aligned(d_m, size_t(size)) || !aligned(d_v, size_t(size))) return fail(RS_EINVAL, "misaligned pointer");
    rs_status st = check_apart({Extent{d_m, adamw->total * size}, Extent{d_v, adamw->total * size}}, {});
    if (st == RS_OK) st = check_ready(adamw);
    if (st == RS_OK) st = check_free(*adamw, d_m, adamw->total * size);
    if (st == RS_OK) st = check_free(*adamw, d_v, adamw->total * size);
    if (st != RS_OK) return st;
    hipError_t e = rs::aw::launch_moments(work_of(*adamw), d_m, d_v, dtype == RS_F32, as_stream(stream));
    if (e != hipSuccess) return hip_fail(e, "adamw moments launch");
    return RS_OK;
}

}  // extern "C"
