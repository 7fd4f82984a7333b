// Group norm on node rows: what etp_abi.cu calls. Internal to libetp.
#pragma once

#include "etp_internal.h"

namespace etp {
namespace norm {

constexpr int kMaxGroups = 64;
constexpr int kMaxVectors = 256;  // of 4, 2 or 1 channels: C at most 1024, 512 or 256
constexpr int kMaxBlocks = 512;   // more than run at once; the workspace holds this many partials

struct Call {
  int lmax, channels, groups, n_nodes, n_structs;
  const int* node_ptr;
  etp_dtype dtype;
  int activation, zero_rest;
};

bool supported(int lmax, int channels, int groups);
// ETP_ERR_BAD_GRAPH unless node_ptr ascends within [0, n_nodes] (synchronises s).
etp_status validate(const Call& c, void* ws, cudaStream_t s);
size_t workspace_bytes(const Call& c, bool backward);
// err: a word on the device or mapped for it that receives the code of a bounded wait that gave up.
etp_status forward(const Call& c, const void* x, const float* weight, const float* bias, float eps, void* out,
                   float* stats, etp_ckpt_format format, uint8_t* q, uint8_t* scale, void* ws, int* err, cudaStream_t s);
etp_status backward(const Call& c, const void* x, etp_ckpt_format format, const uint8_t* q, const uint8_t* scale,
                    const float* stats, const float* weight, const float* bias, const void* grad_out, void* grad_x,
                    float* grad_weight, float* grad_bias, void* ws, int* err, cudaStream_t s);

}  // namespace norm
}  // namespace etp
