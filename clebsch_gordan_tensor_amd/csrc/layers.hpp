// Layers on irreps rows (group norm, dropout, cross attention): handles and launchers.
#pragma once

#include <memory>

#include "cgtp_layers.h"
#include "common.hpp"

namespace cgtp {

// One block of a row: elements [2l+1][mul] from off on; channels counted
// through the blocks from chan on; bias: first bias of a 0e block, else -1.
struct alignas(16) RowBlock {
  int32_t off, nc, mul, chan;
  int32_t bias, chunk, pad0, pad1;  // chunk: first 8-channel chunk (dropout)
};

struct RowLayout {
  std::vector<Irrep> irreps;
  std::vector<RowBlock> blocks;
  int64_t dim = 0, channels = 0, biases = 0, chunks = 0;
};
// Parses and lays out irreps rows (UNSUPPORTED above kLmax or 2^31 elements).
RowLayout row_layout(const char* irreps);

// Device memory owned by a handle, on the device that was current at creation.
class DevMem {
 public:
  DevMem() = default;
  DevMem(const DevMem&) = delete;
  DevMem& operator=(const DevMem&) = delete;
  ~DevMem();
  // Allocates n bytes on the current device and copies them from src (synchronous).
  void upload(const void* src, size_t n);
  void* get() const { return p_; }
  template <typename T>
  const T* as() const { return static_cast<const T*>(p_); }

 private:
  void* p_ = nullptr;
  int device_ = 0;
};

// Most workgroups of 256 threads in one launch, whose threads are counted in 32 bits.
constexpr int64_t kMaxWorkgroups = (int64_t(1) << 24) - 1;

int current_device();
void need_device(int device, const char* what);

// Rows of one sample cut into runs for the norm's kernels.
struct alignas(16) RowChunk {
  int32_t sample, r0, r1, chunk0;  // chunk0: first chunk of the sample
  int32_t nchunk, row0, rows, pad;  // the sample's chunk count, first row and row count
};

// What one workgroup of the norm handles of a block: groups g0 .. g0 + ng - 1,
// at most 256 lanes of `vec` channels (or one larger group).
struct alignas(16) NormStrip {
  int32_t off, nc, mul, chan;  // as RowBlock
  int32_t bias, cg, g0, ng;    // cg: channels per group; g0: first group within the block
  int32_t gid, pad0, pad1, pad2;  // gid: first group over all blocks
};

}  // namespace cgtp

struct cgtp_samples_s {
  int64_t S = 0, rows = 0, nchunk = 0, longest = 0;
  std::vector<int64_t> ptr;
  std::vector<int32_t> sample_chunk;  // host copy: first chunk of each sample, [S + 1]
  int device = 0;
  cgtp::DevMem chunks, first;         // RowChunk [nchunk]; int32 [S + 1] as sample_chunk
  cgtp::DevMem first_row;             // int32 [S + 1] as ptr
};

struct cgtp_norm_s {
  cgtp::RowLayout row;
  int64_t groups = 1, num_groups = 0;
  cgtp_act act = CGTP_ACT_NONE;
  double eps = 0.0;
  cgtp_dtype dtype = CGTP_F32;
  int device = 0;
  // channels per lane: the widest access up to 16 bytes that no group straddles;
  // strips for that width and for single channels (misaligned tensors), then the
  // same as narrow strips (about 128 bytes of channels)
  int vec = 1;
  int64_t narrow_row = 0;  // most elements of a narrow strip in one row
  int nstrip[4] = {0, 0, 0, 0};
  cgtp::DevMem strips[4];
};

struct cgtp_dropout_s {
  cgtp::RowLayout row;
  cgtp_dtype dtype = CGTP_F32;
  int device = 0;
  cgtp::DevMem blocks;
};

namespace cgtp {

size_t norm_ws_bytes(const cgtp_norm_s* n, const cgtp_samples_s* sm, bool backward);
void norm_forward_launch(const cgtp_norm_s* n, const cgtp_samples_s* sm, const void* x, const void* w, const void* b,
                         void* y, void* stats, void* ws, hipStream_t s);
void norm_backward_launch(const cgtp_norm_s* n, const cgtp_samples_s* sm, const void* x, const void* w, const void* b,
                          const void* stats, const void* g, void* gx, void* gw, void* gb, void* ws, hipStream_t s);

void dropout_launch(const cgtp_dropout_s* d, int64_t B, const void* x, double p, uint64_t seed, uint32_t offset,
                    const void* residual, void* y, hipStream_t s);

}  // namespace cgtp
