// ss_ffn_api.cu -- the entry points of the gated feed-forward block
// (include/ss_block.h): argument checks, the workspace, and the launches.
#include <algorithm>

#include "ss_ffn.cuh"

namespace ss {

namespace {

size_t up1024(size_t x) { return (x + 1023) / 1024 * 1024; }

// Workspace: header, then one region that the forward uses for A (when the
// caller keeps none) and the backward for dG, dU and dZ.
struct FfnLayout {
  size_t a, dg, du, dz, total;
};

// Rows of the workspace's [T, F] matrices start on 128-byte boundaries, so that
// no copy of 128 bytes touches a fifth sector and outputs are stored as whole
// sectors whatever F is (backward of T 3001, D 1352, F 3640: 189 -> 172 us).
int64_t workspace_pitch(int64_t F) { return (F + 63) / 64 * 64; }

FfnLayout ffn_layout(int64_t T, int64_t D, int64_t F) {
  FfnLayout L;
  const size_t tf = up1024(static_cast<size_t>(T) * workspace_pitch(F) * 2);
  L.a = L.dg = kHeaderBytes;
  L.du = L.dg + tf;
  L.dz = L.du + tf;
  L.total = L.dz + up1024(static_cast<size_t>(T) * D * 2);
  return L;
}

ss_status check_ffn_sizes(int64_t T, int64_t D, int64_t F) {
  if (T < 0 || D <= 0 || F <= 0) return SS_ERR_INVALID;
  if (T >= (int64_t(1) << 31) || D > SS_MAX_D || F > SS_MAX_F || D % 8 != 0 || F % 8 != 0)
    return SS_ERR_UNSUPPORTED;
  // the tiles are counted in 32 bits
  return T * F < (int64_t(1) << 44) ? SS_OK : SS_ERR_UNSUPPORTED;
}

// every pointer set and 16-byte aligned
bool usable(std::initializer_list<const void*> ps) {
  return std::all_of(ps.begin(), ps.end(), [](const void* p) {
    return p != nullptr && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  });
}

bool low_bits_usable(const void* p) { return reinterpret_cast<uintptr_t>(p) % 32 == 0; }

bool known_act(int act) { return act >= SS_ACT_SILU && act <= SS_ACT_RELU; }

}  // namespace

}  // namespace ss

using namespace ss;

extern "C" {

size_t ss_ffn_workspace_size(int64_t T, int64_t D, int64_t F) {
  return check_ffn_sizes(T, D, F) == SS_OK ? ffn_layout(T, D, F).total : 0;
}

int64_t ss_ffn_low_bits_pitch(int64_t F) { return F > 0 ? (F + 63) / 64 * 64 : 0; }

ss_status ss_ffn_forward(const uint16_t* X, const uint16_t* Wg, const uint16_t* Wu,
                         const uint16_t* Wd, const uint16_t* residual, int64_t T, int64_t D,
                         int64_t F, int act, const ss_dropout_spec* drop, uint16_t* Y, uint16_t* G,
                         uint16_t* U, uint16_t* A, uint8_t* R, void* workspace,
                         size_t workspace_bytes, ss_stream stream) {
  const ss_status st = check_ffn_sizes(T, D, F);
  if (st != SS_OK) return st;
  FfnForward f = {};
  if (!known_act(act) || !make_drop_args(drop, &f.drop)) return SS_ERR_INVALID;
  const bool save = G || U || A;
  if (T > 0 && (!usable({X, Wg, Wu, Wd, Y, workspace}) || (save && !usable({G, U, A})) ||
                (residual && !usable({residual})) || (R && (!save || !low_bits_usable(R)))))
    return SS_ERR_INVALID;
  const FfnLayout L = ffn_layout(T, D, F);
  if (workspace_bytes < L.total) return SS_ERR_WORKSPACE;
  if (T == 0) return SS_OK;
  f.num_sms = current_num_sms();
  if (f.num_sms <= 0)
    return record_failure("cudaGetDevice/cudaDeviceGetAttribute", cudaGetLastError());
  char* ws = static_cast<char*>(workspace);
  f.X = X, f.Wg = Wg, f.Wu = Wu, f.Wd = Wd, f.residual = residual;
  f.T = static_cast<int>(T), f.D = static_cast<int>(D), f.F = static_cast<int>(F), f.act = act;
  f.Y = Y, f.G = G, f.U = U, f.A = save ? A : reinterpret_cast<uint16_t*>(ws + L.a);
  f.ldo = static_cast<int>(save ? F : workspace_pitch(F));
  f.R = R, f.ldr = static_cast<int>(ss_ffn_low_bits_pitch(F));
  f.status = reinterpret_cast<int*>(ws);
  const ForwardPlan plan = forward_plan(T, D, F, f.num_sms);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  {
    StageTrace trace(s, "ffn_gate_up");
    e = plan.up_on_pairs ? pair_gate_up(f, plan.up_pair.bn, s) : split_gate_up(f, plan.up, s);
  }
  if (e != cudaSuccess) return record_failure("ss_ffn_forward (gate/up)", e);
  {
    StageTrace trace(s, "ffn_down");
    e = plan.down_on_pairs ? pair_down(f, s) : split_down(f, plan.down, s);
  }
  return e == cudaSuccess ? SS_OK : record_failure("ss_ffn_forward (down)", e);
}

ss_status ss_ffn_backward(const uint16_t* dY, const uint16_t* X, const uint16_t* Wg,
                          const uint16_t* Wu, const uint16_t* Wd, const uint16_t* G,
                          const uint16_t* U, const uint16_t* A, const uint8_t* R, int64_t T,
                          int64_t D, int64_t F, int act, const ss_dropout_spec* drop, int dw_dtype,
                          int accumulate,
                          uint16_t* dX, void* dWg, void* dWu, void* dWd, void* workspace,
                          size_t workspace_bytes, ss_stream stream) {
  const ss_status st = check_ffn_sizes(T, D, F);
  if (st != SS_OK) return st;
  DropArgs d;
  if (!known_act(act) || !make_drop_args(drop, &d) ||
      (dw_dtype != SS_BF16 && dw_dtype != SS_FP32) || (accumulate != 0 && accumulate != 1))
    return SS_ERR_INVALID;
  if (!usable({dWg, dWu, dWd}) ||
      (T > 0 && (!usable({dY, X, Wg, Wu, Wd, G, U, A, dX, workspace}) ||
                 (R && !low_bits_usable(R)))))
    return SS_ERR_INVALID;
  const FfnLayout L = ffn_layout(T, D, F);
  if (workspace_bytes < L.total) return SS_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    const size_t bytes = static_cast<size_t>(F) * D * (dw_dtype == SS_BF16 ? 2 : 4);
    cudaError_t e = cudaSuccess;
    for (void* w : {dWg, dWu, dWd})
      if (!accumulate && e == cudaSuccess) e = cudaMemsetAsync(w, 0, bytes, s);
    return e == cudaSuccess ? SS_OK : record_failure("ss_ffn_backward (empty batch)", e);
  }
  FfnBackward b = {};
  b.num_sms = current_num_sms();
  if (b.num_sms <= 0)
    return record_failure("cudaGetDevice/cudaDeviceGetAttribute", cudaGetLastError());
  char* ws = static_cast<char*>(workspace);
  uint16_t* dz = reinterpret_cast<uint16_t*>(ws + L.dz);
  b.dZ = d.mode == kDropNone ? dY : dz;
  b.X = X, b.Wg = Wg, b.Wu = Wu, b.Wd = Wd, b.G = G, b.U = U, b.A = A;
  b.T = static_cast<int>(T), b.D = static_cast<int>(D), b.F = static_cast<int>(F), b.act = act;
  b.scale = d.scale;
  b.dw_fp32 = dw_dtype == SS_FP32, b.accumulate = accumulate;
  b.dX = dX, b.dWg = dWg, b.dWu = dWu, b.dWd = dWd;
  b.dG = reinterpret_cast<uint16_t*>(ws + L.dg), b.dU = reinterpret_cast<uint16_t*>(ws + L.du);
  b.ldg = static_cast<int>(workspace_pitch(F));
  b.R = R, b.ldr = static_cast<int>(ss_ffn_low_bits_pitch(F));
  b.status = reinterpret_cast<int*>(ws);
  const BackwardPlan plan = backward_plan(T, D, F, b.num_sms);
  cudaError_t e = cudaSuccess;
  if (d.mode != kDropNone) {
    // zeroes only: the factor 1 / (1 - p) goes into the products' epilogues, so
    // dZ is not rounded a second time
    StageTrace trace(s, "ffn_drop_mask");
    e = launch_drop_mask(dY, T * D, d, dz, b.num_sms, s);
  }
  if (e != cudaSuccess) return record_failure("ss_ffn_backward (mask)", e);
  {
    StageTrace trace(s, "ffn_grad_act");
    e = plan.act_on_pairs ? pair_grad_act(b, plan.act_pair.bn, s) : split_grad_act(b, plan.act, s);
  }
  if (e != cudaSuccess) return record_failure("ss_ffn_backward (dG, dU)", e);
  {
    StageTrace trace(s, "ffn_grads");
    if (plan.grads_together) {
      e = pair_grads(b, kDoX | kDoW, s);
    } else {
      e = plan.x_on_pairs ? pair_grads(b, kDoX, s) : split_grad_x(b, plan.x, s);
      if (e == cudaSuccess)
        e = plan.w_on_pairs ? pair_grads(b, kDoW, s) : split_grad_w(b, plan.w, s);
    }
  }
  return e == cudaSuccess ? SS_OK : record_failure("ss_ffn_backward (dX, dW)", e);
}

}  // extern "C"
