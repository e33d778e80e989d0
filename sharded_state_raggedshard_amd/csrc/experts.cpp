// C-ABI entry points that carry tokens to experts and back: argument checks,
// scratch layout and launches.  Every check happens before the first launch.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <string>

#include "experts.hpp"
#include "raggedshard.h"
#include "row_checks.hpp"

namespace {

using namespace rs::rowcheck;

constexpr int64_t kMaxChoices = 0x7fffffff;
constexpr int32_t kMaxAlign = 1 << 16;

bool sizes_ok(int64_t rows, int32_t experts, int32_t k) {
    return rows >= 0 && experts >= 1 && experts <= rs::kMaxSortExperts && k >= 1 && k <= experts &&
           rows <= kMaxChoices / k;
}

int64_t slots_needed(int64_t rows, int32_t experts, int32_t k, int32_t align) {
    return rows * k + std::min<int64_t>(experts, rows * k) * (align - 1);
}

size_t scratch_bytes(int64_t rows, int32_t experts, int32_t k) {
    const int64_t chunks = std::max<int64_t>(1, rs::sort_chunk_room(rows * k));
    return align256(size_t(chunks) * size_t(experts) * sizeof(int32_t));
}

// Rows of `hidden` values, `rows` of them.
rs_status check_rows(const void* p, int32_t dtype, int64_t rows, int64_t hidden, int64_t ld, bool needed) {
    if (!p && !needed) return RS_OK;
    if (rows > 0 && !p) return fail(RS_EINVAL, "NULL argument");
    if (!aligned(p, dtype == RS_F32 ? 4 : 2)) return fail(RS_EINVAL, "misaligned pointer");
    if (ld < hidden) return fail(RS_EINVAL, "row stride below the row's length");
    if (rows > kMaxElems / ld) return fail(RS_EOVERFLOW, "rows * stride beyond 2^50 elements");
    return RS_OK;
}

// What every call over sorted rows takes, checked and filled in.
rs_status fill(rs::ExpertRows& a, int32_t dtype, int64_t rows, int64_t hidden, const int32_t* slot, int32_t k,
               const float* weight, int64_t ldw, int64_t slots) {
    if (dtype != RS_F32 && dtype != RS_BF16) return fail(RS_EINVAL, "unknown dtype");
    if (rows < 0 || slots < 0) return fail(RS_EINVAL, "negative number of rows");
    if (hidden < 1 || hidden > (int64_t(1) << 24)) return fail(RS_EINVAL, "hidden outside 1..2^24");
    if (k < 1 || k > rs::kMaxSortExperts) return fail(RS_EINVAL, "k outside 1..1024");
    if (rows > kMaxChoices / k || slots > kMaxChoices)
        return fail(RS_EOVERFLOW, "rows * k or slots beyond 2^31 - 1");
    if (rows > 0 && !slot) return fail(RS_EINVAL, "NULL argument");
    if (!aligned(slot, 4) || !aligned(weight, 4)) return fail(RS_EINVAL, "misaligned pointer");
    if (weight && (ldw < k || rows > kMaxElems / ldw)) return fail(RS_EINVAL, "row stride of the weights out of range");
    a = rs::ExpertRows{};
    a.f32 = dtype == RS_F32;
    a.rows = rows;
    a.hidden = hidden;
    a.k = k;
    a.slot = slot;
    a.weight = weight;
    a.ldw = ldw;
    a.slots = slots;
    return RS_OK;
}

rs_status fill_padding(rs::ExpertRows& a, int32_t experts, const int64_t* start, const int32_t* count) {
    if (!start != !count) return fail(RS_EINVAL, "d_start and d_count come together");
    if (!start) return RS_OK;
    if (experts < 1 || experts > rs::kMaxSortExperts) return fail(RS_EINVAL, "experts outside 1..1024");
    if (!aligned(start, 8) || !aligned(count, 4)) return fail(RS_EINVAL, "misaligned pointer");
    a.experts = experts;
    a.start = start;
    a.count = count;
    return RS_OK;
}

Extent slots_of(const rs::ExpertRows& a) { return {a.slot, a.rows * a.k * 4}; }
Extent weights_of(const rs::ExpertRows& a) { return matrix(a.weight, a.rows, a.k, a.ldw, 4); }
Extent starts_of(const rs::ExpertRows& a) { return {a.start, (a.experts + 1) * 8}; }
Extent counts_of(const rs::ExpertRows& a) { return {a.count, a.experts * 4}; }
Extent rows_of(const rs::ExpertRows& a, const void* p, int64_t rows, int64_t ld) {
    return matrix(p, rows, a.hidden, ld, a.f32 ? 4 : 2);
}

}  // namespace

extern "C" {

int64_t rs_expert_slots(int64_t rows, int32_t experts, int32_t k, int32_t align) {
    if (sizes_ok(rows, experts, k) && align >= 1 && align <= kMaxAlign) {
        const int64_t slots = slots_needed(rows, experts, k, align);
        if (slots <= kMaxChoices) return slots;
    }
    fail(RS_EINVAL, "sizes out of range");
    return -1;
}

size_t rs_expert_sort_bytes(int64_t rows, int32_t experts, int32_t k) {
    if (!sizes_ok(rows, experts, k)) {
        fail(RS_EINVAL, "sizes out of range");
        return 0;
    }
    return scratch_bytes(rows, experts, k);
}

rs_status rs_expert_sort(const int64_t* d_topk, int64_t rows, int32_t experts, int32_t k, int64_t ldk,
                         const uint8_t* d_mask, int32_t align, int64_t* d_start, int32_t* d_count, int32_t* d_slot,
                         void* d_work, size_t bytes, void* stream) {
    if (!d_start || !d_count || !d_work) return fail(RS_EINVAL, "NULL argument");
    if (experts < 1 || experts > rs::kMaxSortExperts) return fail(RS_EINVAL, "experts outside 1..1024");
    if (k < 1 || k > experts) return fail(RS_EINVAL, "k outside 1..experts");
    if (rows < 0) return fail(RS_EINVAL, "negative number of rows");
    if (ldk < k) return fail(RS_EINVAL, "row stride below the row's length");
    if (align < 1 || align > kMaxAlign) return fail(RS_EINVAL, "align outside 1..2^16");
    if (rows > kMaxChoices / k || rows > kMaxElems / ldk)
        return fail(RS_EOVERFLOW, "rows * k beyond 2^31 - 1, or rows * ldk beyond 2^50");
    if (slots_needed(rows, experts, k, align) > kMaxChoices)
        return fail(RS_EOVERFLOW, "slots beyond 2^31 - 1");
    if (rows > 0 && (!d_topk || !d_slot)) return fail(RS_EINVAL, "NULL argument");
    if (!aligned(d_topk, 8) || !aligned(d_start, 8) || !aligned(d_count, 4) || !aligned(d_slot, 4))
        return fail(RS_EINVAL, "misaligned pointer");
    if (!aligned(d_work, 16)) return fail(RS_EINVAL, "workspace not 16-byte aligned");
    const size_t need = scratch_bytes(rows, experts, k);
    if (bytes < need)
        return fail(RS_ENOMEM, "workspace of " + std::to_string(bytes) + " bytes; the call needs " + std::to_string(need));
    rs_status st = check_apart({Extent{d_start, (experts + 1) * 8}, Extent{d_count, experts * 4},
                                Extent{d_slot, rows * k * 4}, Extent{d_work, int64_t(need)}},
                               {matrix(d_topk, rows, k, ldk, 8), Extent{d_mask, rows}});
    if (st != RS_OK) return st;
    rs::ExpertSort a;
    a.topk = d_topk;
    a.rows = rows;
    a.ldk = ldk;
    a.experts = experts;
    a.k = k;
    a.align = align;
    a.mask = d_mask;
    a.start = d_start;
    a.count = d_count;
    a.slot = d_slot;
    a.part = static_cast<int32_t*>(d_work);
    hipError_t e = rs::launch_expert_sort(a, as_stream(stream));
    if (e != hipSuccess) return hip_fail(e, "expert_sort launch");
    return RS_OK;
}

rs_status rs_expert_dispatch(const void* d_x, int32_t dtype, int64_t rows, int64_t hidden, int64_t ldx,
                             const int32_t* d_slot, int32_t k, const float* d_weight, int64_t ldw, int32_t experts,
                             const int64_t* d_start, const int32_t* d_count, void* d_y, int64_t slots, int64_t ldy,
                             void* stream) {
    rs::ExpertRows a;
    rs_status st = fill(a, dtype, rows, hidden, d_slot, k, d_weight, ldw, slots);
    if (st == RS_OK) st = fill_padding(a, experts, d_start, d_count);
    if (st == RS_OK) st = check_rows(d_x, dtype, rows, hidden, ldx, true);
    if (st == RS_OK) st = check_rows(d_y, dtype, slots, hidden, ldy, true);
    if (st == RS_OK)
        st = check_apart({rows_of(a, d_y, slots, ldy)},
                         {rows_of(a, d_x, rows, ldx), slots_of(a), weights_of(a), starts_of(a), counts_of(a)});
    if (st != RS_OK) return st;
    hipError_t e = rs::launch_expert_dispatch(a, d_x, ldx, d_y, ldy, as_stream(stream));
    if (e != hipSuccess) return hip_fail(e, "expert_dispatch launch");
    return RS_OK;
}

rs_status rs_expert_combine(const void* d_y, int32_t dtype, int64_t slots, int64_t hidden, int64_t ldy,
                            const int32_t* d_slot, int64_t rows, int32_t k, const float* d_weight, int64_t ldw,
                            const void* d_add, int64_t lda, void* d_out, int64_t ldo, void* stream) {
    rs::ExpertRows a;
    rs_status st = fill(a, dtype, rows, hidden, d_slot, k, d_weight, ldw, slots);
    if (st == RS_OK) st = check_rows(d_y, dtype, slots, hidden, ldy, true);
    if (st == RS_OK) st = check_rows(d_add, dtype, rows, hidden, lda, false);
    if (st == RS_OK) st = check_rows(d_out, dtype, rows, hidden, ldo, true);
    const Extent out = rows_of(a, d_out, rows, ldo);
    if (st == RS_OK) st = check_apart({out}, {rows_of(a, d_y, slots, ldy), slots_of(a), weights_of(a)});
    if (st == RS_OK && !(d_add == d_out && lda == ldo)) st = check_apart({out}, {rows_of(a, d_add, rows, lda)});
    if (st != RS_OK) return st;
    hipError_t e = rs::launch_expert_combine(a, d_y, ldy, d_add, lda, d_out, ldo, as_stream(stream));
    if (e != hipSuccess) return hip_fail(e, "expert_combine launch");
    return RS_OK;
}

rs_status rs_expert_combine_grad(const void* d_dout, int32_t dtype, int64_t rows, int64_t hidden, int64_t ldo,
                                 const void* d_y, int64_t slots, int64_t ldy, const int32_t* d_slot, int32_t k,
                                 const float* d_weight, int64_t ldw, int32_t experts, const int64_t* d_start,
                                 const int32_t* d_count, void* d_dy, int64_t lddy, float* d_dweight, int64_t lddw,
                                 void* stream) {
    rs::ExpertRows a;
    rs_status st = fill(a, dtype, rows, hidden, d_slot, k, d_weight, ldw, slots);
    if (st == RS_OK) st = fill_padding(a, experts, d_start, d_count);
    if (st == RS_OK) st = check_rows(d_dout, dtype, rows, hidden, ldo, true);
    if (st == RS_OK) st = check_rows(d_y, dtype, slots, hidden, ldy, true);
    if (st == RS_OK) st = check_rows(d_dy, dtype, slots, hidden, lddy, false);
    if (st != RS_OK) return st;
    if (rows > 0 && !d_dweight) return fail(RS_EINVAL, "NULL argument");
    if (!aligned(d_dweight, 4)) return fail(RS_EINVAL, "misaligned pointer");
    if (lddw < k || rows > kMaxElems / lddw) return fail(RS_EINVAL, "row stride of the weights' gradient out of range");
    const Extent dy = rows_of(a, d_dy, slots, lddy), dw = matrix(d_dweight, rows, k, lddw, 4);
    st = check_apart({dy, dw}, {rows_of(a, d_dout, rows, ldo), slots_of(a), weights_of(a), starts_of(a), counts_of(a)});
    const Extent y = rows_of(a, d_y, slots, ldy);
    if (st == RS_OK) st = check_apart({dw}, {y});
    if (st == RS_OK && !(d_dy == d_y && lddy == ldy)) st = check_apart({dy}, {y});
    if (st != RS_OK) return st;
    hipError_t e = rs::launch_expert_combine_grad(a, d_dout, ldo, d_y, ldy, d_dy, lddy, d_dweight, lddw, as_stream(stream));
    if (e != hipSuccess) return hip_fail(e, "expert_combine_grad launch");
    return RS_OK;
}

}  // extern "C"
