// Cross attention: argument blocks, work lists, handles.
#pragma once

#include "layers.hpp"

namespace cgtp {
namespace attn {

// 32 consecutive rows: context rows, or query rows (token * G + head in group).
struct Tile {
  int32_t row0, n;
};

// Work of one workgroup: up to four tiles a0 .. a0 + tiles - 1 of one side for
// context head hk, against tiles b0 .. b1 - 1 of the other. slot >= 0: the
// result is part `slot` of a split, at tile slot * stride of the partial buffer;
// tiles = 0: nothing (padding of the list).
struct alignas(16) Item {
  int32_t a0, tiles, b0, b1;
  int32_t hk, slot, stride, kind;  // kind: of gradient items
};
enum : int32_t { kItemQ = 0, kItemV = 1, kItemK = 2 };  // grad_q; grad_v (or both); grad_k

// One tile whose result is the sum of parts slot .. slot + parts - 1, number
// `within` of the `stride` tiles of each.
struct alignas(16) Join {
  int32_t tile, hk, slot, parts;
  int32_t stride, within, pad0, pad1;
};

struct PackTensor {
  const void* src;
  int64_t ld;
  void *row_frags, *col_frags;  // either may be NULL
  bool vec;                     // 16-byte gathers
};

struct PackArgs {
  PackTensor t[2];
  const Tile* tiles;
  const int4* table;
  const uint8_t* mask;  // context rows, or NULL
  const void* out;      // forward's output (for delta)
  int64_t ldo;
  const float* lse;
  float* rows_out;      // queries and grad_out: lse and delta of every row (else NULL)
  float* bias;          // context: 0 or -inf for every key (else NULL)
  float* norms;         // context: largest |k|^2 of every tile and head (or NULL)
  int32_t* flags;       // context: whether a tile has a masked or missing key (or NULL)
  int G, heads, groups;  // G = 0: context rows
  int ntiles, size;  // size: elements of a head
  bool out_vec;
};

// Up to two tensors of equal layout whose parts are added.
struct GradJoinArgs {
  const Join* joins;
  const Tile* tiles;
  const int4* table;
  const float *part0, *part1;
  void *dst0, *dst1;
  int64_t ld;
  int G;  // 1 for context rows
  bool query, quad;
};

struct FwdArgs {
  const Item* items;
  const Join* joins;
  const Tile* qtiles;
  const int4* table;
  const void *q, *kf, *vf;
  const float *bias, *norms;
  const int32_t* flags;
  void* out;
  float *lse, *part;
  float4* part_ml;  // of every row of a part: reference, sum of the rounded weights, of the exact ones
  int64_t ldq, ldo;
  float scale2;     // |scale| log2 e
  uint32_t q_sign;  // flips the queries' signs where the scale is negative
  int G, heads, groups;
  bool q_vec, out_quad;
};

// Packed forms of the gradients: row or column fragments of K, V, Q and grad_out, in
// the order in which they lie in the workspace.
enum : int { kKRows = 0, kVRows = 1, kKCols = 2, kKForms = 3 };
enum : int { kQRows = 0, kGCols = 1, kGRows = 2, kQCols = 3, kQForms = 4 };

struct BwdArgs {
  const Item* items;
  const Tile *qtiles, *ktiles;
  const int4* table;
  // packed forms, one after another at equal strides (in elements)
  const void *kforms_, *qforms_;
  int64_t kstride, qstride;
  template <typename T>
  __host__ __device__ const T* kforms(int form) const {
    return static_cast<const T*>(kforms_) + form * kstride;
  }
  template <typename T>
  __host__ __device__ const T* qforms(int form) const {
    return static_cast<const T*>(qforms_) + form * qstride;
  }
  const float *bias, *rows;
  void *dq, *dk, *dv;
  float *part_q, *part_k, *part_v;
  int64_t ldq, ldk;
  float scale, scale2;
  int G, heads, groups;
  bool q_quad, k_quad;
};

struct KernelTable {
  void (*pack)(const PackArgs&, hipStream_t);
  void (*fwd)(const FwdArgs&, int items, int tiles, hipStream_t);  // items of up to 1, 4 or 8 tiles
  void (*fwd_join)(const FwdArgs&, int joins, hipStream_t);
  void (*bwd)(const BwdArgs&, int items, hipStream_t);  // each gradient unless NULL
  void (*grad_join)(const GradJoinArgs&, int joins, int tensors, hipStream_t);
};

// Kernels of a padded head size (a multiple of 32 up to 256); inst/attn_*.hip.
KernelTable kernels_f32(int dp);
KernelTable kernels_bf16(int dp);

// Whether the forward has a form of 64 query rows a wave (8 tiles an item): its
// operands and accumulators fit the registers.
constexpr bool wide_forward(int dp, size_t size) { return size == 2 && dp <= 128; }

// Whether both gradients of the keys are formed in one pass: their accumulators
// and operands fit the registers (else four products' worth of work becomes five:
// fp32, heads of 128, 3000 queries and 611 keys 231 us in one, 244 us in two).
constexpr bool one_pass(int dp, size_t size) { return dp <= (size == 2 ? 128 : 160); }

// A list of work items on the device with the joins of its splits: those of the
// query side, then those of the context side.
struct WorkList {
  int items = 0, joins[2] = {0, 0};
  int64_t part_tiles[2] = {0, 0};  // tiles of partial results
  DevMem item_mem, join_mem[2];
};

}  // namespace attn
}  // namespace cgtp

struct cgtp_attn_s {
  cgtp::RowLayout qrow, krow;
  int heads = 1, kv_heads = 1, G = 1, D = 0, DP = 0;
  bool vec16 = false, quad = false;  // every head's run is a multiple of 16 bytes / of 4 elements
  cgtp_dtype dtype = CGTP_F32;
  int device = 0;
  cgtp::attn::KernelTable k{};
  cgtp::DevMem table;  // int4 [DP]
};

struct cgtp_attn_batch_s {
  cgtp_attn attn = nullptr;
  int64_t nq = 0, nk = 0;            // rows
  int64_t qtiles = 0, ktiles = 0;
  int device = 0;
  cgtp::DevMem qtile_mem, ktile_mem;
  cgtp::attn::WorkList few, fwd, wide;  // forward, items of up to 1, 4 and 8 query tiles
  cgtp::attn::WorkList bwd;
};

namespace cgtp {

cgtp_attn_s* build_attn(const char* irreps, int64_t heads, int64_t kv_heads, cgtp_dtype dtype);
cgtp_attn_batch_s* build_attn_batch(cgtp_attn_s* at, const cgtp_samples_s* q, const cgtp_samples_s* k);
size_t attn_context_bytes(const cgtp_attn_batch_s* b);
size_t attn_forward_ws_bytes(const cgtp_attn_batch_s* b, bool packed);
size_t attn_backward_ws_bytes(const cgtp_attn_batch_s* b);

struct RowsIn {  // rows with a stride in elements
  const void* p;
  int64_t ld;
};
void attn_pack_launch(const cgtp_attn_batch_s* b, RowsIn k, RowsIn v, const uint8_t* mask, void* context,
                      hipStream_t s);
void attn_forward_launch(const cgtp_attn_batch_s* b, RowsIn q, const void* context, double scale, void* out,
                         float* lse, void* ws, hipStream_t s);
void attn_backward_launch(const cgtp_attn_batch_s* b, RowsIn q, RowsIn k, RowsIn v, const uint8_t* mask, double scale,
                          const void* out, const float* lse, RowsIn g, void* dq, void* dk, void* dv, void* ws,
                          hipStream_t s);

}  // namespace cgtp
