// fa_window.h -- launch interface of the sliding-window kernels (fa_window.cu),
// used by their C entries and by the cache's forward for long query chunks.
#pragma once
#include "fa_launch.h"
#include "fa_win_bwd_kernel.cuh"
#include "fa_win_kernel.cuh"

namespace fa {

// Launches a kernel that begins with grid_dependency_wait() behind the one before it on
// the stream: its blocks are set up while that one still runs.
template <typename... P>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, const P&... p) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kern, p...);
}

struct WinLaunchArgs {
  CUtensorMap tm_q, tm_k, tm_v, tm_o;
  WinParams p;
  int num_sms;
  cudaStream_t stream;
};

// q, o: packed [total_q, H, d] (p.cu_q set) or dense [B, Nq, H, d]; k, v packed
// [total_k, Hk, d], dense [B, Nk, Hk, d], or (kpad) dense with p.cu_k holding
// a length per sequence and Nk a multiple of 128.  Encodes the maps and launches.
int launch_window(WinLaunchArgs& a, const void* q, const void* k, const void* v, int Hk, int d, bool kpad);

// kpad: the workspace for units cut between CTAs, 16-byte aligned.
size_t window_parts_bytes(int num_sms, int d);
void window_parts(WinParams& p, void* at, int num_sms);

}  // namespace fa
