// Group norm on node rows: host side of a call (etp_norm_sweep.h has the kernel).
#include "etp_norm.h"

#include <string>

#include "etp_checkpoint.h"
#include "etp_norm_sweep.h"

namespace etp {
namespace norm {
namespace {

int vector_width(int channels, int groups) {
  const int cg = channels / groups;
  return cg % 4 == 0 ? 4 : cg % 2 == 0 ? 2 : 1;
}

// workspace: [flag of the check of node_ptr][partial sums][means per structure][channel sums per block], the last two
// for the backward
size_t partial_bytes(const Call& c) {
  return align256(static_cast<size_t>(kMaxBlocks) * 2 * (c.lmax + 2) * c.groups * sizeof(double));
}
size_t mean_bytes(const Call& c) {
  return align256(static_cast<size_t>(c.n_structs) * (c.lmax + 2) * c.groups * sizeof(float));
}

__global__ void k_check_ptr(const int* ptr, int n_structs, int n_nodes, int* flag) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i > n_structs) return;
  const int v = ptr[i];
  if (v < 0 || v > n_nodes || (i < n_structs && ptr[i + 1] < v)) *flag = 1;
}

}  // namespace

etp_status validate(const Call& c, void* ws, cudaStream_t s) {
  if (!c.node_ptr) return ETP_OK;
  cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(int), s);
  if (e == cudaSuccess) {
    k_check_ptr<<<c.n_structs / 256 + 1, 256, 0, s>>>(c.node_ptr, c.n_structs, c.n_nodes, static_cast<int*>(ws));
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return cuda_status(e, "node_ptr validation");
  int bad = 0;
  e = cudaMemcpyAsync(&bad, ws, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_status(e, "node_ptr validation");
  if (!bad) return ETP_OK;
  set_error("node_ptr must be ascending and stay within [0, n_nodes]");
  return ETP_ERR_BAD_GRAPH;
}

bool supported(int lmax, int channels, int groups) {
  return lmax >= 0 && lmax <= kMaxL && channels >= 1 && groups >= 1 && groups <= kMaxGroups && channels % groups == 0 &&
         channels / vector_width(channels, groups) <= kMaxVectors && channels * (lmax + 1) * (lmax + 1) <= kGenMaxDim;
}

size_t workspace_bytes(const Call& c, bool backward) {
  size_t n = 256 + partial_bytes(c);
  if (backward) n += mean_bytes(c) + align256(static_cast<size_t>(kMaxBlocks) * (c.lmax + 2) * c.channels * sizeof(float));
  return n;
}

etp_status forward(const Call& c, const void* x, const float* weight, const float* bias, float eps, void* out,
                   float* stats, etp_ckpt_format format, uint8_t* q, uint8_t* scale, void* ws, int* err,
                   cudaStream_t s) {
  Args p{};
  p.ring.src[0] = static_cast<const char*>(x);
  p.weight = weight;
  p.bias = bias;
  p.eps = eps;
  p.act = c.activation;
  p.zero_rest = c.zero_rest;
  p.out = out;
  p.table = stats;
  p.int8 = format == ETP_CKPT_INT8;
  p.err = err;
  p.part = reinterpret_cast<double*>(static_cast<char*>(ws) + 256);
  // the norm writes the checkpoint itself where no block of 32 crosses a component's end
  const bool fused = format != ETP_CKPT_NONE && c.channels % kCkptBlock == 0;
  p.q = fused ? q : nullptr;
  p.scale = fused ? scale : nullptr;
  if (format != ETP_CKPT_NONE && !fused) {
    const int dim = c.channels * (c.lmax + 1) * (c.lmax + 1);
    etp_status st = ckpt::store(format, c.dtype, c.n_nodes, dim, x, q, scale, s);
    if (st != ETP_OK) return st;
  }
  const int width = vector_width(c.channels, c.groups);
  return launch_forward(c, p, width, s);
}

etp_status backward(const Call& c, const void* x, etp_ckpt_format format, const uint8_t* q, const uint8_t* scale,
                    const float* stats, const float* weight, const float* bias, const void* grad_out, void* grad_x,
                    float* grad_weight, float* grad_bias, void* ws, int* err, cudaStream_t s) {
  const bool kept = format != ETP_CKPT_NONE;
  Args p{};
  p.ring.src[0] = static_cast<const char*>(grad_out);
  p.ring.src[1] = kept ? reinterpret_cast<const char*>(q) : static_cast<const char*>(x);
  p.ring.src[2] = reinterpret_cast<const char*>(scale);
  p.int8 = format == ETP_CKPT_INT8;
  p.stats_in = stats;
  p.weight = weight;
  p.bias = bias;
  p.act = c.activation;
  p.zero_rest = c.zero_rest;
  p.out = grad_x;
  p.grad_weight = grad_weight;
  p.grad_bias = grad_bias;
  p.err = err;
  char* at = static_cast<char*>(ws) + 256;
  p.part = reinterpret_cast<double*>(at);
  p.table = reinterpret_cast<float*>(at += partial_bytes(c));
  p.chan = reinterpret_cast<float*>(at + mean_bytes(c));
  // Of 32-bit rows the backward takes two channels a thread, of 16-bit rows four. Two keep a row in work for
  // half as long and the sums in registers; four share a row's addresses, scales and codes among more
  // values, but at rank 3 from a checkpoint they spill (272 to 304 bytes). Two / four channels, us, 8
  // structures, 128 channels, 65.5 MB of float32 rows (or their values in bfloat16), from rows, int8, e4m3:
  //            float32                               bfloat16
  //   rank 1   52.0/52.1  45.4/42.9  45.5/41.7       36.6/33.0  43.0/37.0  43.1/36.2
  //   rank 2   53.3/55.0  42.0/42.0  42.0/41.6       32.4/30.6  37.5/34.7  37.6/33.8
  //   rank 3   53.6/56.4  43.3/48.3  43.1/47.5       31.5/31.0  36.2/41.3  36.3/39.6
  // The type alone is not the best rule for rank 1 in 32 bits and rank 3 in 16 bits from checkpoints.
  int width = vector_width(c.channels, c.groups);
  if (c.dtype == ETP_F32 && width == 4 && c.channels / 2 <= kMaxVectors) width = 2;
  return launch_backward(c, p, kept, width, s);
}

}  // namespace norm
}  // namespace etp
