// C-ABI entry points (include/ep.h): host-side validation, workspace sizing
// and kernel launches.  Nothing here touches the device before validation
// has passed, and nothing here allocates.
#include "ep.h"
#include "ep_internal.h"

#include <atomic>
#include <mutex>

// Device scratch of ep_layout_dispatch_static: the workspace of callers that
// cannot allocate.  Every GPU the library runs on holds its own copy until
// the process ends.  In host code `scratch` names a host-side stand-in, not a
// device address: only the pointer that hipGetSymbolAddress returns for the
// current device may reach a kernel or a copy.
static __device__ __align__(256) unsigned char scratch[EP_STATIC_SCRATCH_BYTES];

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 31;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shape checks shared by the layout and dispatch calls.
ep_status_t check_routing_shape(int32_t T, int32_t K, int32_t E, int32_t P) {
    if (T < 0 || K <= 0 || E <= 0 || P <= 0) return EP_ERR_INVALID_ARG;
    if (E % P != 0 || K > E) return EP_ERR_INVALID_ARG;
    if ((int64_t)T * K >= kMaxRows) return EP_ERR_INVALID_ARG;
    if (E > EP_MAX_EXPERTS || K > EP_MAX_TOPK) return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

ep_status_t from_hip(hipError_t e) { return e == hipSuccess ? EP_OK : EP_ERR_HIP; }

// Address of the current device's copy of `scratch`, looked up once per
// device (with that device current) and kept.
constexpr int kScratchDevices = 64;
std::atomic<void*> g_scratch_ptr[kScratchDevices];
std::mutex g_scratch_mu;

ep_status_t device_scratch(void** out) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return EP_ERR_HIP;
    if (dev < 0 || dev >= kScratchDevices) return EP_ERR_UNSUPPORTED;
    void* p = g_scratch_ptr[dev].load(std::memory_order_acquire);
    if (!p) {
        std::lock_guard<std::mutex> lock(g_scratch_mu);
        p = g_scratch_ptr[dev].load(std::memory_order_acquire);
        if (!p) {
            if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p)
                return EP_ERR_HIP;
            g_scratch_ptr[dev].store(p, std::memory_order_release);
        }
    }
    *out = p;
    return EP_OK;
}

}  // namespace

extern "C" {

size_t ep_workspace_bytes(int32_t num_tokens, int32_t num_topk, int32_t num_experts,
                          int32_t num_partitions) {
    if (check_routing_shape(num_tokens, num_topk, num_experts, num_partitions) != EP_OK)
        return 0;
    return ep::ws_map(num_tokens, num_topk, num_experts, num_partitions).total;
}

ep_status_t ep_get_dispatch_layout(const int64_t* topk_idx, int32_t num_tokens,
                                   int32_t num_topk, int32_t num_experts,
                                   int32_t num_partitions, int32_t* num_tokens_per_expert,
                                   int32_t* num_tokens_per_partition,
                                   uint8_t* is_token_in_partition, int32_t* expert_offsets,
                                   int32_t* partition_offsets, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    const int32_t T = num_tokens, K = num_topk, E = num_experts, P = num_partitions;
    ep_status_t st = check_routing_shape(T, K, E, P);
    if (st != EP_OK) return st;
    if (!num_tokens_per_expert || !num_tokens_per_partition || !expert_offsets ||
        !partition_offsets || !workspace)
        return EP_ERR_INVALID_ARG;
    if (T > 0 && (!topk_idx || !is_token_in_partition)) return EP_ERR_INVALID_ARG;
    const ep::WsMap m = ep::ws_map(T, K, E, P);
    if (workspace_bytes < m.total) return EP_ERR_WORKSPACE;
    return from_hip(ep::launch_layout(topk_idx, T, K, E, P, workspace, m, num_tokens_per_expert,
                                      num_tokens_per_partition, is_token_in_partition,
                                      expert_offsets, partition_offsets,
                                      static_cast<hipStream_t>(stream)));
}

ep_status_t ep_dispatch(const void* x, int32_t num_tokens, int32_t hidden,
                        const int64_t* topk_idx, int32_t num_topk, int32_t num_experts,
                        int32_t num_partitions, ep_dtype_t out_dtype, void* recv_x,
                        float* recv_scales, int32_t* recv_src_token, int32_t* dst_row,
                        const void* workspace, size_t workspace_bytes, void* stream) {
    const int32_t T = num_tokens, H = hidden, K = num_topk, E = num_experts, P = num_partitions;
    ep_status_t st = check_routing_shape(T, K, E, P);
    if (st != EP_OK) return st;
    if (out_dtype != EP_DTYPE_BF16 && out_dtype != EP_DTYPE_FP8_E4M3) return EP_ERR_INVALID_ARG;
    const bool fp8 = out_dtype == EP_DTYPE_FP8_E4M3;
    if (H <= 0 || H % 8 != 0 || (fp8 && H % 128 != 0)) return EP_ERR_INVALID_ARG;
    if (!workspace) return EP_ERR_INVALID_ARG;
    if (T > 0) {
        if (!x || !topk_idx || !recv_x || !recv_src_token || !dst_row) return EP_ERR_INVALID_ARG;
        if (fp8 && !recv_scales) return EP_ERR_INVALID_ARG;
        if (!aligned16(x) || !aligned16(recv_x)) return EP_ERR_INVALID_ARG;
    }
    const ep::WsMap m = ep::ws_map(T, K, E, P);
    if (workspace_bytes < m.total) return EP_ERR_WORKSPACE;
    return from_hip(ep::launch_dispatch(static_cast<const uint16_t*>(x), T, H, K, fp8, recv_x,
                                        recv_scales, recv_src_token, dst_row, workspace, m, 0,
                                        T * K, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// Argument checks of the one-call layout + dispatch (the workspace apart).
ep_status_t check_layout_dispatch(const void* x, int32_t T, int32_t H, const int64_t* topk_idx,
                                  int32_t K, int32_t E, int32_t P, ep_dtype_t out_dtype,
                                  const int32_t* num_tokens_per_expert,
                                  const int32_t* num_tokens_per_partition,
                                  const uint8_t* is_token_in_partition,
                                  const int32_t* expert_offsets, const int32_t* partition_offsets,
                                  const void* recv_x, const float* recv_scales,
                                  const int32_t* recv_src_token, const int32_t* dst_row) {
    ep_status_t st = check_routing_shape(T, K, E, P);
    if (st != EP_OK) return st;
    if (out_dtype != EP_DTYPE_BF16 && out_dtype != EP_DTYPE_FP8_E4M3) return EP_ERR_INVALID_ARG;
    const bool fp8 = out_dtype == EP_DTYPE_FP8_E4M3;
    if (H <= 0 || H % 8 != 0 || (fp8 && H % 128 != 0)) return EP_ERR_INVALID_ARG;
    if (!num_tokens_per_expert || !num_tokens_per_partition || !expert_offsets ||
        !partition_offsets)
        return EP_ERR_INVALID_ARG;
    if (T > 0) {
        if (!x || !topk_idx || !is_token_in_partition || !recv_x || !recv_src_token || !dst_row)
            return EP_ERR_INVALID_ARG;
        if (fp8 && !recv_scales) return EP_ERR_INVALID_ARG;
        if (!aligned16(x) || !aligned16(recv_x)) return EP_ERR_INVALID_ARG;
    }
    return EP_OK;
}

}  // namespace

extern "C" {

ep_status_t ep_layout_dispatch_cu(const void* x, int32_t num_tokens, int32_t hidden,
                                  const int64_t* topk_idx, int32_t num_topk, int32_t num_experts,
                                  int32_t num_partitions, ep_dtype_t out_dtype,
                                  int32_t* num_tokens_per_expert,
                                  int32_t* num_tokens_per_partition,
                                  uint8_t* is_token_in_partition, int32_t* expert_offsets,
                                  int32_t* partition_offsets, void* recv_x, float* recv_scales,
                                  int32_t* recv_src_token, int32_t* dst_row, void* workspace,
                                  size_t workspace_bytes, int32_t num_cus, void* stream) {
    const int32_t T = num_tokens, H = hidden, K = num_topk, E = num_experts, P = num_partitions;
    ep_status_t st = check_layout_dispatch(x, T, H, topk_idx, K, E, P, out_dtype,
                                           num_tokens_per_expert, num_tokens_per_partition,
                                           is_token_in_partition, expert_offsets,
                                           partition_offsets, recv_x, recv_scales,
                                           recv_src_token, dst_row);
    if (st != EP_OK) return st;
    if (!workspace || num_cus < 0) return EP_ERR_INVALID_ARG;
    const bool fp8 = out_dtype == EP_DTYPE_FP8_E4M3;
    const ep::WsMap m = ep::ws_map(T, K, E, P);
    if (workspace_bytes < m.total) return EP_ERR_WORKSPACE;
    return from_hip(ep::launch_layout_dispatch(
        static_cast<const uint16_t*>(x), topk_idx, T, H, K, E, P, fp8, workspace, m,
        num_tokens_per_expert, num_tokens_per_partition, is_token_in_partition, expert_offsets,
        partition_offsets, recv_x, recv_scales, recv_src_token, dst_row, num_cus,
        static_cast<hipStream_t>(stream)));
}

ep_status_t ep_layout_dispatch(const void* x, int32_t num_tokens, int32_t hidden,
                               const int64_t* topk_idx, int32_t num_topk, int32_t num_experts,
                               int32_t num_partitions, ep_dtype_t out_dtype,
                               int32_t* num_tokens_per_expert, int32_t* num_tokens_per_partition,
                               uint8_t* is_token_in_partition, int32_t* expert_offsets,
                               int32_t* partition_offsets, void* recv_x, float* recv_scales,
                               int32_t* recv_src_token, int32_t* dst_row, void* workspace,
                               size_t workspace_bytes, void* stream) {
    return ep_layout_dispatch_cu(x, num_tokens, hidden, topk_idx, num_topk, num_experts,
                                 num_partitions, out_dtype, num_tokens_per_expert,
                                 num_tokens_per_partition, is_token_in_partition, expert_offsets,
                                 partition_offsets, recv_x, recv_scales, recv_src_token, dst_row,
                                 workspace, workspace_bytes, 0, stream);
}

ep_status_t ep_layout_dispatch_static(const void* x, int32_t num_tokens, int32_t hidden,
                                      const int64_t* topk_idx, int32_t num_topk,
                                      int32_t num_experts, int32_t num_partitions,
                                      ep_dtype_t out_dtype, int32_t* num_tokens_per_expert,
                                      int32_t* num_tokens_per_partition,
                                      uint8_t* is_token_in_partition, int32_t* expert_offsets,
                                      int32_t* partition_offsets, void* recv_x,
                                      float* recv_scales, int32_t* recv_src_token,
                                      int32_t* dst_row, void* stream) {
    const int32_t T = num_tokens, H = hidden, K = num_topk, E = num_experts, P = num_partitions;
    ep_status_t st = check_layout_dispatch(x, T, H, topk_idx, K, E, P, out_dtype,
                                           num_tokens_per_expert, num_tokens_per_partition,
                                           is_token_in_partition, expert_offsets,
                                           partition_offsets, recv_x, recv_scales,
                                           recv_src_token, dst_row);
    if (st != EP_OK) return st;
    if (ep::ws_map(T, K, E, P).total > (size_t)EP_STATIC_SCRATCH_BYTES) return EP_ERR_UNSUPPORTED;
    void* ws = nullptr;
    st = device_scratch(&ws);
    if (st != EP_OK) return st;
    // The kernels and outputs of ep_layout_dispatch, with the device's scratch
    // as the workspace.  Nothing in it needs clearing: every layout call
    // writes all that its dispatch launch reads.
    return ep_layout_dispatch_cu(x, num_tokens, hidden, topk_idx, num_topk, num_experts,
                                 num_partitions, out_dtype, num_tokens_per_expert,
                                 num_tokens_per_partition, is_token_in_partition, expert_offsets,
                                 partition_offsets, recv_x, recv_scales, recv_src_token, dst_row,
                                 ws, (size_t)EP_STATIC_SCRATCH_BYTES, 0, stream);
}

int64_t ep_aligned_rows(int32_t num_tokens, int32_t num_topk, int32_t num_experts,
                        int32_t expert_alignment) {
    if (check_routing_shape(num_tokens, num_topk, num_experts, 1) != EP_OK) return 0;
    if (expert_alignment < 1 || expert_alignment > EP_MAX_EXPERT_ALIGNMENT) return 0;
    const int64_t R = (int64_t)num_tokens * num_topk +
                      (int64_t)num_experts * (expert_alignment - 1);
    return R < kMaxRows ? R : 0;
}

ep_status_t ep_layout_dispatch_aligned(const void* x, int32_t num_tokens, int32_t hidden,
                                       const int64_t* topk_idx, int32_t num_topk,
                                       int32_t num_experts, int32_t num_partitions,
                                       int32_t expert_alignment, ep_dtype_t out_dtype,
                                       int32_t* num_tokens_per_expert,
                                       int32_t* num_tokens_per_partition,
                                       uint8_t* is_token_in_partition, int32_t* expert_offsets,
                                       int32_t* partition_offsets, void* recv_x,
                                       float* recv_scales, int32_t* recv_src_token,
                                       int32_t* dst_row, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    const int32_t T = num_tokens, H = hidden, K = num_topk, E = num_experts, P = num_partitions;
    ep_status_t st = check_routing_shape(T, K, E, P);
    if (st != EP_OK) return st;
    const int64_t R = ep_aligned_rows(T, K, E, expert_alignment);
    if (R == 0 && T > 0) return EP_ERR_INVALID_ARG;
    if (expert_alignment < 1 || expert_alignment > EP_MAX_EXPERT_ALIGNMENT)
        return EP_ERR_INVALID_ARG;
    if (out_dtype != EP_DTYPE_BF16 && out_dtype != EP_DTYPE_FP8_E4M3) return EP_ERR_INVALID_ARG;
    const bool fp8 = out_dtype == EP_DTYPE_FP8_E4M3;
    if (H <= 0 || H % 8 != 0 || (fp8 && H % 128 != 0)) return EP_ERR_INVALID_ARG;
    if (!num_tokens_per_expert || !num_tokens_per_partition || !expert_offsets ||
        !partition_offsets || !workspace)
        return EP_ERR_INVALID_ARG;
    if (R > 0 && !recv_src_token) return EP_ERR_INVALID_ARG;
    if (T > 0) {
        if (!x || !topk_idx || !is_token_in_partition || !recv_x || !dst_row)
            return EP_ERR_INVALID_ARG;
        if (fp8 && !recv_scales) return EP_ERR_INVALID_ARG;
        if (!aligned16(x) || !aligned16(recv_x)) return EP_ERR_INVALID_ARG;
    }
    const ep::WsMap m = ep::ws_map(T, K, E, P);
    if (workspace_bytes < m.total) return EP_ERR_WORKSPACE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = ep::launch_layout_aligned(topk_idx, T, K, E, P, expert_alignment, workspace, m,
                                             num_tokens_per_expert, num_tokens_per_partition,
                                             is_token_in_partition, expert_offsets,
                                             partition_offsets, recv_src_token, R, s);
    if (e != hipSuccess) return EP_ERR_HIP;
    return from_hip(ep::launch_dispatch(static_cast<const uint16_t*>(x), T, H, K, fp8, recv_x,
                                        recv_scales, recv_src_token, dst_row, workspace, m, 0,
                                        (int)R, s));
}

ep_status_t ep_dispatch_dedup(const void* x, int32_t num_tokens, int32_t hidden,
                              const int64_t* topk_idx, int32_t num_topk, int32_t num_experts,
                              int32_t num_partitions, ep_dtype_t out_dtype,
                              int32_t* num_tokens_per_expert, int32_t* num_tokens_per_partition,
                              uint8_t* is_token_in_partition, int32_t* expert_offsets,
                              int32_t* partition_offsets, int32_t* partition_token_offsets,
                              void* recv_x, float* recv_scales, int32_t* recv_src_token,
                              int32_t* recv_topk_idx, int32_t* slot_src_row, int32_t* dst_row,
                              void* workspace, size_t workspace_bytes, void* stream) {
    const int32_t T = num_tokens, H = hidden, K = num_topk, E = num_experts, P = num_partitions;
    ep_status_t st = check_routing_shape(T, K, E, P);
    if (st != EP_OK) return st;
    if (out_dtype != EP_DTYPE_BF16 && out_dtype != EP_DTYPE_FP8_E4M3) return EP_ERR_INVALID_ARG;
    const bool fp8 = out_dtype == EP_DTYPE_FP8_E4M3;
    if (H <= 0 || H % 8 != 0 || (fp8 && H % 128 != 0)) return EP_ERR_INVALID_ARG;
    if (!num_tokens_per_expert || !num_tokens_per_partition || !expert_offsets ||
        !partition_offsets || !partition_token_offsets || !workspace)
        return EP_ERR_INVALID_ARG;
    if (T > 0) {
        if (!x || !topk_idx || !is_token_in_partition || !recv_x || !recv_src_token ||
            !recv_topk_idx || !slot_src_row || !dst_row)
            return EP_ERR_INVALID_ARG;
        if (fp8 && !recv_scales) return EP_ERR_INVALID_ARG;
        if (!aligned16(x) || !aligned16(recv_x)) return EP_ERR_INVALID_ARG;
    }
    const ep::WsMap m = ep::ws_map(T, K, E, P);
    if (workspace_bytes < m.total) return EP_ERR_WORKSPACE;
    return from_hip(ep::launch_dispatch_dedup(
        static_cast<const uint16_t*>(x), topk_idx, T, H, K, E, P, fp8, workspace, m,
        num_tokens_per_expert, num_tokens_per_partition, is_token_in_partition, expert_offsets,
        partition_offsets, partition_token_offsets, recv_x, recv_scales, recv_src_token,
        recv_topk_idx, slot_src_row, dst_row, static_cast<hipStream_t>(stream)));
}

ep_status_t ep_low_latency_dispatch(const void* x, int32_t num_tokens, int32_t hidden,
                                    const int64_t* topk_idx, int32_t num_topk,
                                    int32_t num_experts, int32_t capacity, ep_dtype_t out_dtype,
                                    int32_t* num_tokens_per_expert, void* recv_x,
                                    float* recv_scales, int32_t* recv_src_token,
                                    int32_t* dst_row, int64_t* num_invalid, void* stream) {
    const int32_t T = num_tokens, H = hidden, K = num_topk, E = num_experts, C = capacity;
    ep_status_t st = check_routing_shape(T, K, E, 1);
    if (st != EP_OK) return st;
    if (C <= 0 || (int64_t)E * C >= kMaxRows) return EP_ERR_INVALID_ARG;
    if (out_dtype != EP_DTYPE_BF16 && out_dtype != EP_DTYPE_FP8_E4M3) return EP_ERR_INVALID_ARG;
    const bool fp8 = out_dtype == EP_DTYPE_FP8_E4M3;
    if (H <= 0 || H % 8 != 0 || (fp8 && H % 128 != 0)) return EP_ERR_INVALID_ARG;
    if (!num_tokens_per_expert || !recv_src_token) return EP_ERR_INVALID_ARG;
    if (T > 0) {
        if (!x || !topk_idx || !recv_x || !dst_row) return EP_ERR_INVALID_ARG;
        if (fp8 && !recv_scales) return EP_ERR_INVALID_ARG;
        if (!aligned16(x) || !aligned16(recv_x)) return EP_ERR_INVALID_ARG;
    }
    if ((int64_t)T * K > EP_LL_MAX_SLOTS) return EP_ERR_UNSUPPORTED;
    return from_hip(ep::launch_ll_dispatch(
        static_cast<const uint16_t*>(x), topk_idx, T, H, K, E, C, fp8, num_tokens_per_expert,
        recv_x, recv_scales, recv_src_token, dst_row, num_invalid,
        static_cast<hipStream_t>(stream)));
}

ep_status_t ep_combine_cu(const void* y, int64_t num_rows, const int32_t* dst_row,
                          const float* topk_weights, int32_t num_tokens, int32_t num_topk,
                          int32_t hidden, void* out, int32_t num_cus, void* stream) {
    const int32_t T = num_tokens, K = num_topk, H = hidden;
    if (T < 0 || K <= 0 || H <= 0 || H % 8 != 0 || num_rows < 0 || num_cus < 0)
        return EP_ERR_INVALID_ARG;
    if ((int64_t)T * K >= kMaxRows) return EP_ERR_INVALID_ARG;
    if (K > EP_MAX_TOPK || H > EP_MAX_COMBINE_HIDDEN) return EP_ERR_UNSUPPORTED;
    if (T > 0) {
        if (!dst_row || !topk_weights || !out) return EP_ERR_INVALID_ARG;
        if ((y && !aligned16(y)) || !aligned16(out)) return EP_ERR_INVALID_ARG;
    }
    if (T > 0 && num_rows > 0 && !y) return EP_ERR_INVALID_ARG;
    return from_hip(ep::launch_combine(static_cast<const uint16_t*>(y), num_rows, dst_row,
                                       topk_weights, T, K, H, static_cast<uint16_t*>(out),
                                       num_cus, static_cast<hipStream_t>(stream)));
}

ep_status_t ep_combine(const void* y, int64_t num_rows, const int32_t* dst_row,
                       const float* topk_weights, int32_t num_tokens, int32_t num_topk,
                       int32_t hidden, void* out, void* stream) {
    return ep_combine_cu(y, num_rows, dst_row, topk_weights, num_tokens, num_topk, hidden, out, 0,
                         stream);
}

ep_status_t ep_combine_backward(const void* grad_out, const void* y, int64_t num_rows,
                                const int32_t* dst_row, const float* topk_weights,
                                int32_t num_tokens, int32_t num_topk, int32_t hidden,
                                void* grad_y, float* grad_weights, void* stream) {
    const int32_t T = num_tokens, K = num_topk, H = hidden;
    if (T < 0 || K <= 0 || H <= 0 || H % 8 != 0 || num_rows < 0) return EP_ERR_INVALID_ARG;
    if ((int64_t)T * K >= kMaxRows) return EP_ERR_INVALID_ARG;
    if (K > EP_MAX_TOPK || H > EP_MAX_COMBINE_HIDDEN) return EP_ERR_UNSUPPORTED;
    if (T > 0) {
        // without rows every slot is skipped: grad_y and y may then be empty
        if (!grad_out || !dst_row) return EP_ERR_INVALID_ARG;
        if (!grad_weights && !grad_y && num_rows > 0) return EP_ERR_INVALID_ARG;
        if (grad_y && !topk_weights) return EP_ERR_INVALID_ARG;
        if (grad_weights && num_rows > 0 && !y) return EP_ERR_INVALID_ARG;
        if (!aligned16(grad_out) || (y && !aligned16(y)) || (grad_y && !aligned16(grad_y)))
            return EP_ERR_INVALID_ARG;
    }
    return from_hip(ep::launch_combine_backward(
        static_cast<const uint16_t*>(grad_out),
        grad_weights ? static_cast<const uint16_t*>(y) : nullptr, num_rows, dst_row, topk_weights,
        T, K, H, static_cast<uint16_t*>(grad_y), grad_weights,
        static_cast<hipStream_t>(stream)));
}

ep_status_t ep_dispatch_backward(const void* grad_recv_x, int64_t num_rows,
                                 const int32_t* dst_row, int32_t num_tokens, int32_t num_topk,
                                 int32_t hidden, void* grad_x, void* stream) {
    const int32_t T = num_tokens, K = num_topk, H = hidden;
    if (T < 0 || K <= 0 || H <= 0 || H % 8 != 0 || num_rows < 0) return EP_ERR_INVALID_ARG;
    if ((int64_t)T * K >= kMaxRows) return EP_ERR_INVALID_ARG;
    if (K > EP_MAX_TOPK || H > EP_MAX_COMBINE_HIDDEN) return EP_ERR_UNSUPPORTED;
    if (T > 0) {
        if (!dst_row || !grad_x || (num_rows > 0 && !grad_recv_x)) return EP_ERR_INVALID_ARG;
        if ((grad_recv_x && !aligned16(grad_recv_x)) || !aligned16(grad_x))
            return EP_ERR_INVALID_ARG;
    }
    return from_hip(ep::launch_combine(static_cast<const uint16_t*>(grad_recv_x), num_rows,
                                       dst_row, nullptr, T, K, H,
                                       static_cast<uint16_t*>(grad_x), 0,
                                       static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// Shape and type checks shared by the router and its gradient.
ep_status_t check_route(ep_dtype_t dtype, int32_t T, int32_t E, int32_t K, ep_score_t score,
                        float scale) {
    if (T < 0 || E <= 0 || K <= 0 || K > E) return EP_ERR_INVALID_ARG;
    if (dtype != EP_DTYPE_BF16 && dtype != EP_DTYPE_FP32) return EP_ERR_INVALID_ARG;
    if (score != EP_SCORE_SOFTMAX && score != EP_SCORE_SIGMOID) return EP_ERR_INVALID_ARG;
    if (!(scale - scale == 0.0f)) return EP_ERR_INVALID_ARG;   // infinite or NaN
    if ((int64_t)T * K >= kMaxRows) return EP_ERR_INVALID_ARG;
    if (E > EP_MAX_EXPERTS || K > EP_MAX_TOPK) return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

extern "C" {

ep_status_t ep_route(const void* logits, ep_dtype_t logits_dtype, const float* expert_bias,
                     int32_t num_tokens, int32_t num_experts, int32_t num_topk, ep_score_t score,
                     int32_t num_groups, int32_t topk_groups, int32_t normalize, float scale,
                     int64_t* topk_idx, float* topk_weights, void* stream) {
    const int32_t T = num_tokens, E = num_experts, K = num_topk;
    ep_status_t st = check_route(logits_dtype, T, E, K, score, scale);
    if (st != EP_OK) return st;
    if (num_groups < 1 || E % num_groups != 0 || topk_groups < 1 || topk_groups > num_groups ||
        (int64_t)K > (int64_t)topk_groups * (E / num_groups))
        return EP_ERR_INVALID_ARG;
    if (num_groups > EP_MAX_ROUTE_GROUPS) return EP_ERR_UNSUPPORTED;
    const bool bf16 = logits_dtype == EP_DTYPE_BF16;
    if (T > 0) {
        if (!logits || !topk_idx || !topk_weights) return EP_ERR_INVALID_ARG;
        if (!aligned_to(logits, bf16 ? 2 : 4)) return EP_ERR_INVALID_ARG;
    }
    return from_hip(ep::launch_route(logits, bf16, expert_bias, T, E, K,
                                     score == EP_SCORE_SOFTMAX, num_groups, topk_groups,
                                     normalize != 0, scale, topk_idx, topk_weights,
                                     static_cast<hipStream_t>(stream)));
}

ep_status_t ep_route_backward(const void* logits, ep_dtype_t logits_dtype,
                              const int64_t* topk_idx, const float* grad_weights,
                              int32_t num_tokens, int32_t num_experts, int32_t num_topk,
                              ep_score_t score, int32_t normalize, float scale,
                              void* grad_logits, void* stream) {
    const int32_t T = num_tokens, E = num_experts, K = num_topk;
    ep_status_t st = check_route(logits_dtype, T, E, K, score, scale);
    if (st != EP_OK) return st;
    const bool bf16 = logits_dtype == EP_DTYPE_BF16;
    if (T > 0) {
        if (!logits || !topk_idx || !grad_weights || !grad_logits) return EP_ERR_INVALID_ARG;
        if (!aligned_to(logits, bf16 ? 2 : 4) || !aligned_to(grad_logits, bf16 ? 2 : 4))
            return EP_ERR_INVALID_ARG;
    }
    return from_hip(ep::launch_route_backward(logits, bf16, topk_idx, grad_weights, T, E, K,
                                              score == EP_SCORE_SOFTMAX, normalize != 0, scale,
                                              grad_logits, static_cast<hipStream_t>(stream)));
}

ep_status_t ep_expert_linear_w4(const void* x, const float* x_scales, ep_dtype_t x_dtype,
                                int64_t num_rows, const int32_t* expert_offsets,
                                const int32_t* num_tokens_per_expert, int32_t capacity,
                                int32_t num_experts, int32_t in_features, int32_t out_features,
                                int32_t group_size, const uint8_t* weight, const void* scales,
                                const uint8_t* zeros, int32_t swiglu, void* y, void* stream) {
    const int32_t E = num_experts, I = in_features, N = out_features, G = group_size;
    if (E <= 0 || I <= 0 || N <= 0 || N % 8 != 0 || num_rows < 0 || num_rows >= kMaxRows)
        return EP_ERR_INVALID_ARG;
    if ((G != 32 && G != 64 && G != 128) || I % G != 0) return EP_ERR_INVALID_ARG;
    if (x_dtype != EP_DTYPE_BF16 && x_dtype != EP_DTYPE_FP8_E4M3) return EP_ERR_INVALID_ARG;
    const bool fp8 = x_dtype == EP_DTYPE_FP8_E4M3;
    if (fp8 && I % 128 != 0) return EP_ERR_INVALID_ARG;
    if (!expert_offsets && (capacity < 1 || (int64_t)E * capacity > num_rows))
        return EP_ERR_INVALID_ARG;
    if (num_rows > 0) {
        if (!x || !num_tokens_per_expert || !weight || !scales || !y || (fp8 && !x_scales))
            return EP_ERR_INVALID_ARG;
        if (!aligned16(x) || !aligned16(weight) || !aligned16(y) || !aligned_to(scales, 8) ||
            !aligned_to(zeros, 4))
            return EP_ERR_INVALID_ARG;
    }
    const int64_t W = (int64_t)N * (swiglu ? 2 : 1);
    if (E > EP_MAX_EXPERTS || I > EP_MAX_EXPERT_IN || W * (I / 2) >= kMaxRows)
        return EP_ERR_UNSUPPORTED;
    return from_hip(ep::launch_expert_linear_w4(
        x, x_scales, fp8, num_rows, expert_offsets, num_tokens_per_expert, capacity, E, I, N, G,
        weight, static_cast<const uint16_t*>(scales), zeros, swiglu != 0,
        static_cast<uint16_t*>(y), static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// The checks that the calls over the experts' rows share.
ep_status_t check_runs(int64_t num_rows, const int32_t* offsets, const int32_t* counts,
                       int32_t capacity, int32_t E) {
    if (E <= 0 || num_rows < 0 || num_rows >= kMaxRows) return EP_ERR_INVALID_ARG;
    if (!offsets && (capacity < 1 || (int64_t)E * capacity > num_rows)) return EP_ERR_INVALID_ARG;
    if (!counts) return EP_ERR_INVALID_ARG;
    return E > EP_MAX_EXPERTS ? EP_ERR_UNSUPPORTED : EP_OK;
}

}  // namespace

extern "C" {

ep_status_t ep_expert_linear(const void* x, const float* x_scales, ep_dtype_t dtype,
                             int64_t num_rows, const int32_t* expert_offsets,
                             const int32_t* num_tokens_per_expert, int32_t capacity,
                             int32_t num_experts, int32_t in_features, int32_t out_features,
                             const void* weight, const float* weight_scales, int32_t swiglu,
                             void* y, void* stream) {
    const int32_t E = num_experts, I = in_features, N = out_features;
    if (dtype != EP_DTYPE_BF16 && dtype != EP_DTYPE_FP8_E4M3) return EP_ERR_INVALID_ARG;
    const bool fp8 = dtype == EP_DTYPE_FP8_E4M3;
    if (I <= 0 || I % (fp8 ? 128 : 8) != 0 || N <= 0 || N % 8 != 0) return EP_ERR_INVALID_ARG;
    if (num_rows > 0) {
        if (!x || !weight || !y || (fp8 && (!x_scales || !weight_scales)))
            return EP_ERR_INVALID_ARG;
        if (!aligned16(x) || !aligned16(weight) || !aligned16(y)) return EP_ERR_INVALID_ARG;
    }
    ep_status_t st = check_runs(num_rows, expert_offsets, num_tokens_per_expert, capacity, E);
    if (st != EP_OK) return st;
    if (I > EP_MAX_LINEAR_CHANNELS || (int64_t)N * (swiglu ? 2 : 1) > EP_MAX_LINEAR_CHANNELS)
        return EP_ERR_UNSUPPORTED;
    const ep::RowRuns runs = {expert_offsets, num_tokens_per_expert, capacity, E, num_rows};
    return from_hip(ep::launch_expert_linear(x, fp8 ? x_scales : nullptr, runs, I, N, weight,
                                             weight_scales, swiglu != 0,
                                             static_cast<uint16_t*>(y),
                                             static_cast<hipStream_t>(stream)));
}

ep_status_t ep_expert_linear_backward(const void* grad_y, const void* x, const void* weight,
                                      int64_t num_rows, const int32_t* expert_offsets,
                                      const int32_t* num_tokens_per_expert, int32_t capacity,
                                      int32_t num_experts, int32_t in_features,
                                      int32_t out_features, void* grad_x, void* grad_weight,
                                      ep_dtype_t grad_weight_dtype, int32_t accumulate,
                                      void* stream) {
    const int32_t E = num_experts, I = in_features, N = out_features;
    if (I <= 0 || I % 8 != 0 || N <= 0 || N % 8 != 0) return EP_ERR_INVALID_ARG;
    const bool fp32 = grad_weight_dtype == EP_DTYPE_FP32;
    if (grad_weight && !fp32 && (grad_weight_dtype != EP_DTYPE_BF16 || accumulate))
        return EP_ERR_INVALID_ARG;
    if (!grad_x && !grad_weight) return EP_ERR_INVALID_ARG;
    if (grad_weight && !aligned16(grad_weight)) return EP_ERR_INVALID_ARG;
    if (num_rows > 0) {
        if (!grad_y || !aligned16(grad_y)) return EP_ERR_INVALID_ARG;
        if (grad_x && (!weight || !aligned16(weight) || !aligned16(grad_x)))
            return EP_ERR_INVALID_ARG;
        if (grad_weight && (!x || !aligned16(x))) return EP_ERR_INVALID_ARG;
    }
    ep_status_t st = check_runs(num_rows, expert_offsets, num_tokens_per_expert, capacity, E);
    if (st != EP_OK) return st;
    if (I > EP_MAX_LINEAR_CHANNELS || N > EP_MAX_LINEAR_CHANNELS) return EP_ERR_UNSUPPORTED;
    const ep::RowRuns runs = {expert_offsets, num_tokens_per_expert, capacity, E, num_rows};
    return from_hip(ep::launch_expert_gradients(
        static_cast<const uint16_t*>(grad_y), static_cast<const uint16_t*>(x), runs, I, N,
        static_cast<const uint16_t*>(weight), static_cast<uint16_t*>(grad_x), grad_weight, fp32,
        accumulate != 0, static_cast<hipStream_t>(stream)));
}

ep_status_t ep_expert_swiglu(const void* gate_up, int64_t num_rows, const int32_t* expert_offsets,
                             const int32_t* num_tokens_per_expert, int32_t capacity,
                             int32_t num_experts, int32_t features, ep_dtype_t out_dtype, void* y,
                             float* y_scales, void* stream) {
    const int32_t E = num_experts, N = features;
    if (out_dtype != EP_DTYPE_BF16 && out_dtype != EP_DTYPE_FP8_E4M3) return EP_ERR_INVALID_ARG;
    const bool fp8 = out_dtype == EP_DTYPE_FP8_E4M3;
    if (N <= 0 || N % (fp8 ? 128 : 8) != 0 || num_rows < 0 || num_rows >= kMaxRows)
        return EP_ERR_INVALID_ARG;
    if (num_rows > 0) {
        if (!gate_up || !y || (fp8 && !y_scales)) return EP_ERR_INVALID_ARG;
        if (!aligned16(gate_up) || !aligned16(y)) return EP_ERR_INVALID_ARG;
    }
    if (num_tokens_per_expert) {
        ep_status_t st = check_runs(num_rows, expert_offsets, num_tokens_per_expert, capacity, E);
        if (st != EP_OK) return st;
    }
    if (N > EP_MAX_LINEAR_CHANNELS) return EP_ERR_UNSUPPORTED;
    const ep::RowRuns runs = {expert_offsets, num_tokens_per_expert, capacity, E, num_rows};
    return from_hip(ep::launch_expert_swiglu(
        static_cast<const uint16_t*>(gate_up), runs, N, fp8 ? nullptr : static_cast<uint16_t*>(y),
        fp8 ? static_cast<uint8_t*>(y) : nullptr, y_scales, static_cast<hipStream_t>(stream)));
}

ep_status_t ep_expert_swiglu_backward(const void* grad_y, const void* gate_up, int64_t num_rows,
                                      const int32_t* expert_offsets,
                                      const int32_t* num_tokens_per_expert, int32_t capacity,
                                      int32_t num_experts, int32_t features, void* grad_gate_up,
                                      void* stream) {
    const int32_t E = num_experts, N = features;
    if (N <= 0 || N % 8 != 0 || num_rows < 0 || num_rows >= kMaxRows) return EP_ERR_INVALID_ARG;
    if (num_rows > 0) {
        if (!grad_y || !gate_up || !grad_gate_up) return EP_ERR_INVALID_ARG;
        if (!aligned16(grad_y) || !aligned16(gate_up) || !aligned16(grad_gate_up))
            return EP_ERR_INVALID_ARG;
    }
    if (num_tokens_per_expert) {
        ep_status_t st = check_runs(num_rows, expert_offsets, num_tokens_per_expert, capacity, E);
        if (st != EP_OK) return st;
    }
    if (N > EP_MAX_LINEAR_CHANNELS) return EP_ERR_UNSUPPORTED;
    const ep::RowRuns runs = {expert_offsets, num_tokens_per_expert, capacity, E, num_rows};
    return from_hip(ep::launch_expert_swiglu_backward(
        static_cast<const uint16_t*>(grad_y), static_cast<const uint16_t*>(gate_up), runs, N,
        static_cast<uint16_t*>(grad_gate_up), static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// Shape and type checks shared by the norm and its gradient.
ep_status_t check_norm(ep_dtype_t weight_dtype, const void* weight, int32_t T, int32_t H) {
    if (T < 0 || H <= 0 || H % 8 != 0) return EP_ERR_INVALID_ARG;
    if (weight_dtype != EP_DTYPE_BF16 && weight_dtype != EP_DTYPE_FP32) return EP_ERR_INVALID_ARG;
    if (T > 0 && (!weight || !aligned16(weight))) return EP_ERR_INVALID_ARG;
    return H > EP_MAX_NORM_HIDDEN ? EP_ERR_UNSUPPORTED : EP_OK;
}

}  // namespace

extern "C" {

ep_status_t ep_rms_norm(const void* x, const void* residual, const void* weight,
                        ep_dtype_t weight_dtype, int32_t num_tokens, int32_t hidden, float eps,
                        void* y, uint8_t* codes, float* scales, void* residual_out,
                        float* inv_rms, void* stream) {
    const int32_t T = num_tokens, H = hidden;
    ep_status_t st = check_norm(weight_dtype, weight, T, H);
    if (st == EP_ERR_INVALID_ARG) return st;
    if (!(eps >= 0.0f && eps - eps == 0.0f)) return EP_ERR_INVALID_ARG;
    if (T > 0) {
        if (!x || !aligned16(x) || (!y && !codes)) return EP_ERR_INVALID_ARG;
        if (y && !aligned16(y)) return EP_ERR_INVALID_ARG;
        if (codes && (!scales || !aligned16(codes))) return EP_ERR_INVALID_ARG;
        if (!residual != !residual_out) return EP_ERR_INVALID_ARG;
        if (residual && (!aligned16(residual) || !aligned16(residual_out)))
            return EP_ERR_INVALID_ARG;
    }
    if (codes && H % 128 != 0) return EP_ERR_INVALID_ARG;
    if (st != EP_OK || T == 0) return st;
    return from_hip(ep::launch_rms_norm(
        static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(residual), weight,
        weight_dtype == EP_DTYPE_FP32, T, H, eps, static_cast<uint16_t*>(y), codes, scales,
        static_cast<uint16_t*>(residual_out), inv_rms, static_cast<hipStream_t>(stream)));
}

size_t ep_rms_norm_backward_workspace_bytes(int32_t num_tokens, int32_t hidden) {
    if (check_norm(EP_DTYPE_FP32, nullptr, 0, hidden) != EP_OK || num_tokens < 0) return 0;
    return (size_t)(ep::norm_parts(num_tokens) > 0 ? ep::norm_parts(num_tokens) : 1) * hidden *
           sizeof(float);
}

ep_status_t ep_rms_norm_backward(const void* grad_y, const void* x, const void* weight,
                                 ep_dtype_t weight_dtype, const float* inv_rms,
                                 const void* grad_residual, int32_t num_tokens, int32_t hidden,
                                 void* grad_x, float* grad_weight, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    const int32_t T = num_tokens, H = hidden;
    ep_status_t st = check_norm(weight_dtype, weight, T, H);
    if (st != EP_OK) return st;
    if (!grad_weight || !aligned16(grad_weight) || !workspace || !aligned16(workspace))
        return EP_ERR_INVALID_ARG;
    if (T > 0) {
        if (!grad_y || !x || !inv_rms || !grad_x) return EP_ERR_INVALID_ARG;
        if (!aligned16(grad_y) || !aligned16(x) || !aligned16(grad_x)) return EP_ERR_INVALID_ARG;
        if (grad_residual && !aligned16(grad_residual)) return EP_ERR_INVALID_ARG;
    }
    if (workspace_bytes < ep_rms_norm_backward_workspace_bytes(T, H)) return EP_ERR_WORKSPACE;
    return from_hip(ep::launch_rms_norm_backward(
        static_cast<const uint16_t*>(grad_y), static_cast<const uint16_t*>(x), weight,
        weight_dtype == EP_DTYPE_FP32, inv_rms, static_cast<const uint16_t*>(grad_residual), T, H,
        static_cast<uint16_t*>(grad_x), grad_weight, static_cast<float*>(workspace),
        static_cast<hipStream_t>(stream)));
}

ep_status_t ep_get_device_error(const void* workspace, size_t workspace_bytes,
                                int64_t* num_invalid, void* stream) {
    if (!workspace || !num_invalid || workspace_bytes < ep::kWsHeaderBytes)
        return EP_ERR_INVALID_ARG;
    const ep::WsHeader* hdr = static_cast<const ep::WsHeader*>(workspace);
    hipStream_t s = static_cast<hipStream_t>(stream);
    int64_t v = 0;
    if (hipMemcpyAsync(&v, &hdr->num_invalid, sizeof v, hipMemcpyDeviceToHost, s) !=
        hipSuccess)
        return EP_ERR_HIP;
    if (hipStreamSynchronize(s) != hipSuccess) return EP_ERR_HIP;
    *num_invalid = v;
    return EP_OK;
}

const char* ep_status_string(ep_status_t status) {
    switch (status) {
        case EP_OK: return "EP_OK";
        case EP_ERR_INVALID_ARG: return "EP_ERR_INVALID_ARG";
        case EP_ERR_UNSUPPORTED: return "EP_ERR_UNSUPPORTED";
        case EP_ERR_WORKSPACE: return "EP_ERR_WORKSPACE";
        case EP_ERR_HIP: return "EP_ERR_HIP";
    }
    return "EP_ERR_UNKNOWN";
}

ep_status_t ep_convert_e4m3(const float* in, uint8_t* out, int64_t n, int32_t mode,
                            void* stream) {
    if (n < 0 || (n > 0 && (!in || !out)) || (mode != 0 && mode != 1)) return EP_ERR_INVALID_ARG;
    return from_hip(ep::launch_convert_e4m3(in, out, n, mode, static_cast<hipStream_t>(stream)));
}

ep_status_t ep_convert_bf16(const float* in, uint16_t* out, int64_t n, void* stream) {
    if (n < 0 || (n > 0 && (!in || !out))) return EP_ERR_INVALID_ARG;
    return from_hip(ep::launch_convert_bf16(in, out, n, static_cast<hipStream_t>(stream)));
}

ep_status_t ep_copy(const void* src, void* dst, size_t bytes, void* stream) {
    if (bytes % 16 != 0) return EP_ERR_INVALID_ARG;
    if (bytes > 0 && (!src || !dst || !aligned16(src) || !aligned16(dst)))
        return EP_ERR_INVALID_ARG;
    return from_hip(ep::launch_copy(src, dst, bytes, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
