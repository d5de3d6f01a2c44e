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

// What the queries of a tile see of their sample's context. Key tiles are numbered
// through the packed context: first those of the rows that all samples share, then
// every sample's own. Work lists count the key tiles of a sample's queries on from 0:
// tile t stands for t + (t < shared ? 0 : skip). In a causal batch query token i sees
// the places (32 * tile + row within) of its own keys below i + shift.
struct Reach {
  int32_t skip, shift;
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
  int32_t* bad;         // whether a tile and head holds an infinity or NaN (SeqTable::pack)
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
  const Reach* reach;  // of every query tile (sequence kernels only, as the next two)
  int shared;          // key tiles of shared rows
  bool causal;
};

// How a step's places are shared out. A turn is a tile of 32 keys for each of the waves of a
// head; the turns of all slots (those of a slot with several tiles of query rows one tile
// after another) lie end to end, and workgroup i of `shares` takes the i-th stretch of
// max(min_turns, turns / shares). Slots of any lengths so keep all workgroups busy alike.
// Tile of rows e gets its results from consecutive workgroups, one part each, and part
// (i, e) is number i + e: the pairs go along a staircase, so no two are alike.
struct StepCut {
  const int32_t* lengths;  // NULL: no step
  int slots, capacity, tiles_a_slot, waves_a_head, shares, min_turns;
  // turns before every slot and in all, [slots + 1], written by SeqTable::step_sums where
  // there are many slots; NULL: every wave adds the lengths up itself
  int32_t* before;
};
// Slots from which a kernel of its own adds the lengths up; else every workgroup of the step and of
// the join reads all of them (us with and without, 4 heads of 128 in bf16, up to 120 tokens a slot: 128
// slots 29.7 and 29.1, 256 slots 38.5 and 41.8, 1024 slots 82 and 194, 4096 slots 278 and 2115).
constexpr int kStepSumSlots = 256;

// Joins the results of rows against their own context (`own`: the parts of its joins, or
// of a step) with those against rows that all samples share (parts of tiles of 32
// consecutive rows whatever their sample: unit u = per tiles, parts of unit u and context
// head hk from slot (hk * units + u) * parts on).
struct RowsJoinArgs {
  FwdArgs own;
  const float* part;  // of the shared rows, with their references and sums
  const float4* part_ml;
  int units, per, parts;     // parts = 0: nothing is shared
  StepCut cut;
};

// Waves of a step's workgroup: what its shared memory holds of their keys and values.
constexpr int step_waves(int dp, size_t size) { return dp * int(size) <= 512 ? 4 : 2; }

// Whether one launch takes a step and its rows against the shared ones.
constexpr bool step_with_joint(int dp, size_t size) { return step_waves(dp, size) == 4; }

// Channels of a context row next to each other: elements off + head * cw on, with the first head of the
// workgroup for `head`, are elements d on of the workgroup's head j.
struct alignas(16) StepPiece {
  int32_t off, cw, j, d;
};

// One token a slot on caches of rows [slot][capacity][dim].
struct StepArgs {
  FwdArgs f;
  FwdArgs joint;     // against the shared rows: in workgroups of the same launch
  int joint_blocks;  // (a multiple of 8; 0: none, or launched before), of which this many are items
  int joint_items;
  StepCut cut;
  const void *k_new, *v_new;
  int64_t ldk, ldv;
  void *k_cache, *v_cache;
  int64_t dim;
  int size;                            // elements of a head
  int heads_a_group, bundles, pieces;  // heads of a workgroup; workgroups of a row's heads; pieces of a row for them
  const StepPiece* piece;
  int width;    // channels of a piece
  bool whole;   // a workgroup takes a whole tile of rows (no shares): rows are final
  bool joined;  // rows are joined with those against shared rows: all results are parts
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
  const Reach* reach;  // as in FwdArgs
  int shared;
  bool causal;
  const int32_t *k_bad, *q_bad;  // causal: tiles and heads that hold an infinity or NaN
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

// Kernels of batches with shared rows or causal queries, and of steps on a cache;
// inst/attn_seq_*.hip.
struct SeqTable {
  void (*pack)(const PackArgs&, hipStream_t);  // for the gradients of causal batches
  void (*fwd)(const FwdArgs&, int items, int tiles, hipStream_t);
  void (*bwd)(const BwdArgs&, int items, hipStream_t);
  void (*step_sums)(const StepCut&, hipStream_t);
  void (*step)(const StepArgs&, hipStream_t);
  void (*rows_join)(const RowsJoinArgs&, int joins, hipStream_t);
  // of `count` query tiles (with the key tiles that they see), for every context head; NULL in fp32
  void (*delta)(const BwdArgs&, const int4* tiles, int count, float* rows, hipStream_t);
};
SeqTable seq_kernels_f32(int dp);
SeqTable seq_kernels_bf16(int dp);

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

// All query rows of several samples in tiles of 32, whatever their sample, against the
// rows that the samples share; every result is a part.
struct JointPlan {
  int per = 0, units = 0, parts = 0;  // as RowsJoinArgs; per = 0: none
  DevMem tiles;
  WorkList list;
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
  cgtp::attn::SeqTable seq{};
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
  bool causal = false, sequence = false;  // sequence: causal, or with shared rows
  int64_t shared_tiles = 0;
  cgtp::DevMem reach;                 // Reach [qtiles]
  cgtp::attn::JointPlan joint;        // used where every sample has few rows
  int few_keys = 0;                   // query tiles that see few keys
  cgtp::DevMem few_keys_mem;          // int4 [few_keys]: as SeqTable::delta takes them
};

struct cgtp_attn_cache_s {
  cgtp_attn attn = nullptr;
  int64_t slots = 0, capacity = 0, shared = 0, shared_tiles = 0, qtiles = 0;
  int device = 0;
  int heads_a_group = 1, waves_a_head = 1, bundles = 1, tiles_a_slot = 1, shares = 1, min_turns = 1;
  bool whole = false;
  int joins = 0;
  int width[3] = {0, 0, 0}, pieces[3] = {0, 0, 0};  // channels of a piece (0: none such), pieces of a row
  cgtp::DevMem qtile_mem, shared_tile_mem, join_mem, piece_mem[3];
  cgtp::attn::JointPlan joint;
};

namespace cgtp {

cgtp_attn_s* build_attn(const char* irreps, int64_t heads, int64_t kv_heads, cgtp_dtype dtype);
cgtp_attn_batch_s* build_attn_batch(cgtp_attn_s* at, const cgtp_samples_s* q, const cgtp_samples_s* k, bool causal,
                                    int64_t shared);
cgtp_attn_cache_s* build_attn_cache(cgtp_attn_s* at, int64_t slots, int64_t capacity, int64_t shared);
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
size_t attn_cache_shared_bytes(const cgtp_attn_cache_s* c);
size_t attn_step_ws_bytes(const cgtp_attn_cache_s* c);
void attn_share_launch(const cgtp_attn_cache_s* c, RowsIn k, RowsIn v, const uint8_t* mask, void* context,
                       hipStream_t s);
void attn_step_launch(const cgtp_attn_cache_s* c, RowsIn q, RowsIn k, RowsIn v, void* k_cache, void* v_cache,
                      const int32_t* lengths, const void* context, double scale, void* out, float* lse, void* ws,
                      hipStream_t s);
void attn_backward_launch(const cgtp_attn_batch_s* b, RowsIn q, RowsIn k, RowsIn v, const uint8_t* mask, double scale,
                          const void* out, const float* lse, RowsIn g, void* dq, void* dk, void* dv, void* ws,
                          hipStream_t s);

}  // namespace cgtp
