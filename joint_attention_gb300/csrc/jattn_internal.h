// jattn_internal.h — declarations shared by the libjattn translation units
// (kernel launchers and their parameter blocks).  Host-side only; no torch.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace jattn {

// Launches kernel<<<grid, block, smem, st>>>(args...) with programmatic
// stream serialisation, so that its launch and prologue overlap the tail of
// the previous kernel on the stream (the kernel waits on griddepcontrol.wait
// before reading its inputs).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// The same with thread-block clusters of `cluster` CTAs (1: none).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), int cluster, dim3 grid, dim3 block, size_t smem,
                               cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Tile sizes of the tensor-core kernels: 128 query rows per tile (the
// tcgen05 M = 128 accumulator, one row per TMEM lane), 128 keys per tile.
constexpr int kTileM = 128;
constexpr int kTileN = 128;

// Rows of every head split into segments that attend only within
// themselves.  A [B, H, N, d] call is B*H heads of one segment [0, N); a
// packed variable-length call is H heads of T = sum of the sequence lengths
// rows with one segment per sequence.  Segment s holds the head's rows
// [cu[s], cu[s+1]); in the 128-row-padded per-head scratch (-LSE log2 e and
// D for the attention backward) it starts at pcu[s], so pcu[s+1] - pcu[s] is
// 128 times the segment's number of 128-row tiles.
constexpr int kMaxSegments = 256;
struct SegTable {
  int n;      // segments per head (1 .. kMaxSegments)
  int rows;   // rows per head
  int prows;  // padded rows per head (pcu[n])
  int cu[kMaxSegments + 1];
  int pcu[kMaxSegments + 1];
};
// Fills t from n + 1 row offsets (cu[0] = 0, strictly increasing); false if
// they are not valid or n is out of range.
bool make_seg_table(SegTable* t, const int* cu, int n);
// One segment of N rows (the [B, H, N, d] layout).
void make_uniform_seg_table(SegTable* t, int N);

// --- norm / elementwise kernels (HBM-bound) ---------------------------------
// The streaming norm kernels take the per-launch device error word: their
// bounded waits on the bulk-copy ring report a timeout through it.
// rq / rk (1/rms of every q / k row) are written unless null.
cudaError_t launch_qk_norm_fwd(const uint16_t* q, const uint16_t* k, const float* gq, const float* gk,
                               uint16_t* qhat, uint16_t* khat, float* rq, float* rk, int64_t rows, int d,
                               uint32_t* dev_err, cudaStream_t st);
// Rows are the BH heads' seg.rows rows.  The softmax statistics are written
// in the per-head padded layout (segment s from seg.pcu[s], 128-row
// multiples): `stats` gets 16 bf16 per row, -LSE * inv_scale and -D each as
// three bf16 terms whose sum rounds to the fp32 value (columns 0-2 and 3-5;
// pad rows -1e30 and 0), zeros after.  The
// dq accumulator rows are zeroed unless dqacc is null (the deterministic
// backward stores its first contribution); the first n_tickets words of
// `tickets` are zeroed.  With qhat null (q_hat, k_hat, rq and rk saved by a
// training forward) only the statistics, the zeroing and the tickets are
// done, and q, k, qhat, khat, rq, rk are not accessed.  With zero_count
// non-null, the zeroing is skipped when *zero_count == zeroed_by (a training
// forward's CTAs zeroed the accumulator and counted themselves there).
cudaError_t launch_bwd_prep(const uint16_t* q, const uint16_t* k, const float* gq, const float* gk,
                            const uint16_t* out, const uint16_t* dout, const float* lse, uint16_t* qhat,
                            uint16_t* khat, float* rq, float* rk, uint16_t* stats,
                            float inv_scale, float* dqacc, unsigned int* tickets, int n_tickets, int BH,
                            const SegTable& seg, int d, uint32_t* dev_err, cudaStream_t st,
                            const uint32_t* zero_count = nullptr, uint32_t zeroed_by = 0);
// nparts = q_norm_bwd_parts() CTAs, each writing one d-vector of dgq
// partials; the last one (by *ticket, zeroed by the backward preparation)
// sums them and the nk dgk partials into dgq and dgk.  zero_count (or null)
// is reset to 0: the accumulator it vouched for is no longer zero.
cudaError_t launch_q_norm_bwd(const float* dqacc, const uint16_t* q, const float* rq, const float* gq, float scale,
                              uint16_t* dq, float* dgq_part, int nparts, int64_t rows, const float* dgk_part, int nk,
                              unsigned int* ticket, float* dgq, float* dgk, int d, uint32_t* dev_err,
                              cudaStream_t st, uint32_t* zero_count = nullptr);
int q_norm_bwd_parts(int d);
// Streaming multiprocessors of the current device (cached after the first
// call), or the limit set by set_sm_limit if that is lower: the number of
// CTAs the persistent kernels launch.
int device_sm_count();
void set_sm_limit(int n);  // n <= 0: no limit

// --- token-row norm kernels (HBM-bound) ---------------------------------------
// h = bf16(x + res), r = (mean h^2 + eps)^(-1/2), z = g h r; y = bf16(z), or
// y8 = e4m3(448 z / m) with the rows' scales s = m / 448, m = max |z| (the quotient
// rounded to fp32 first).  g null (and y null): z = x.
struct TokenNorm {
  const uint16_t *x, *res;  // res: or null (then h is null)
  const float* g;
  int T, C;  // C a multiple of 8, at most JATTN_MAX_WIDTH
  float eps;
  uint16_t *h, *y;
  uint8_t* y8;
  float *s, *r;  // r: or null
};
cudaError_t launch_add_norm(const TokenNorm& t, cudaStream_t st);
// add_norm_bwd_parts(T, C) blocks, each writing C partial sums of dg to part;
// launch_dg_sum adds them in a fixed order.
int add_norm_bwd_parts(int T, int C);
cudaError_t launch_add_norm_bwd(const uint16_t* dy, const uint16_t* dh, const uint16_t* h, const float* r,
                                const float* g, int T, int C, uint16_t* dx, float* part, int parts,
                                cudaStream_t st);
cudaError_t launch_dg_sum(const float* part, int parts, int C, float* dg, cudaStream_t st);

// LayerNorm: h = bf16(x + res), mu = mean h, r = (mean (h - mu)^2 + eps)^(-1/2),
// y = bf16(g (h - mu) r + b), with gain and bias rows of `items` equal runs of rows.
struct LayerNorm {
  const uint16_t *x, *res;  // res: or null (then h is null)
  const float *g, *b;       // [items, C]; b: or null
  int items, T, C;          // T a multiple of items; C as above
  float eps;
  uint16_t *h, *y;
  float *mean, *r;  // or null
};
cudaError_t launch_layer_norm(const LayerNorm& t, cudaStream_t st);
struct LayerNormBwd {
  const uint16_t *dy, *dh, *h;  // dh: or null
  const float *mean, *r, *g;
  int items, T, C;
  uint16_t* dx;
  float *dg, *db;  // [items, C]; db: or null
};
// layer_norm_bwd_parts(items, T, C) blocks an item, each writing C partial sums of
// dg, and of db if there is one, to part; launch_layer_norm_sums adds an item's in a
// fixed order.
int layer_norm_bwd_parts(int items, int T, int C);
cudaError_t launch_layer_norm_bwd(const LayerNormBwd& t, float* part, int parts, cudaStream_t st);
cudaError_t launch_layer_norm_sums(const float* part, int parts, const LayerNormBwd& t, cudaStream_t st);

// --- rotary positions (HBM-bound) ---------------------------------------------
constexpr int kMaxAxes = 4;
struct Rope {
  int B, Hq, Hk, N, d;  // q [B, Hq, N, d], k [B, Hk, N, d]
  const float* pos;     // [N, axes], or with per_item [B, N, axes]
  bool per_item;
  const float* freq;    // [sum of pairs]
  int axes, pairs[kMaxAxes];
  bool interleaved;
  const float *gq, *gk;  // [d] gains of the QK-RMSNorm, or both null
  float eps;
};
// backward: the rotation's transpose (no gains).
cudaError_t launch_rope(const Rope& t, const uint16_t* q, const uint16_t* k, uint16_t* q_out, uint16_t* k_out,
                        bool backward, cudaStream_t st);
// With gains: part holds d partial sums for each of rope_bwd_parts blocks, of_q of q
// and the others of k, which launch_rope_gains adds in a fixed order.
int64_t rope_bwd_parts(const Rope& t, int64_t* of_q);
cudaError_t launch_rope_norm_bwd(const Rope& t, const uint16_t* dq_rot, const uint16_t* dk_rot, const uint16_t* q,
                                 const uint16_t* k, uint16_t* dq, uint16_t* dk, float* part, cudaStream_t st);
cudaError_t launch_rope_gains(const Rope& t, const float* part, float* dgq, float* dgk, cudaStream_t st);

// --- tensor-core attention kernels ------------------------------------------
struct AttnShape {
  int BH;        // heads (B*H, or H for a packed variable-length call)
  int N;         // rows per head
  int d;
  float scale;   // 1/sqrt(d)
  SegTable seg;  // the heads' segments (one segment [0, N) for the [B, H, N, d] layout)
  bool deterministic = false;  // backward: fixed dQ accumulation order
};

// dq_zero / zero_count (training pair, else null): the backward's fp32 dQ
// accumulator ([BH, rows, d]) to zero, and the word each CTA increments once
// its share is zeroed (attn_fwd_grid(s) increments in all).
cudaError_t launch_attn_fwd(const CUtensorMap& map_q, const CUtensorMap& map_k, const CUtensorMap& map_v,
                            const AttnShape& s, uint16_t* out, float* lse, uint32_t* dev_err, cudaStream_t st,
                            float* dq_zero = nullptr, uint32_t* zero_count = nullptr);
int attn_fwd_grid(const AttnShape& s);

// Packed sequences with grouped heads: q [Hq, T, d], k and v [Hk, T, d] as they are (no
// norm), causal or not.  seg: the sequences that have rows (seg.rows = T, which may lie
// behind the last one).
struct GroupedShape {
  int Hq, Hk, T, d;
  bool causal;
  float scale;
  bool deterministic;  // backward: fixed dQ accumulation order
  SegTable seg;
};
cudaError_t launch_attn_fwd_grouped(const GroupedShape& s, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                    uint16_t* out, float* lse, uint32_t* dev_err, cudaStream_t st);
// Parts that a kv head's query heads are split into where few heads and long sequences
// would leave CTAs idle (1: not split; a divisor of Hq / Hk); a function of the shape alone.
int grouped_parts(const GroupedShape& s);
// Whether no sequence has more than a tile's 128 rows: launch_attn_bwd_grouped then writes dq itself.
bool grouped_direct(const GroupedShape& s);
// The statistics (as launch_bwd_prep's); zeroes dqacc [Hq, T, d] (null: not; rows of the sequences) and
// counters, one word per 128 padded rows of a query head (null: not).
cudaError_t launch_grouped_prep(const GroupedShape& s, const uint16_t* out, const uint16_t* dout, const float* lse,
                                uint16_t* stats, float* dqacc, uint32_t* counters, cudaStream_t st);
// After launch_grouped_prep (with dqacc unless grouped_direct).  With parts > 1 dk and dv go to part, fp32
// [parts][dk, dv][Hk, T, d], and launch_grouped_join adds the parts in order; launch_grouped_round
// makes dq of dqacc (unless grouped_direct).
cudaError_t launch_attn_bwd_grouped(const GroupedShape& s, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                    const uint16_t* dout, const uint16_t* stats, float* dqacc, uint32_t* counters,
                                    uint16_t* dq, uint16_t* dk, uint16_t* dv, float* part, int parts,
                                    uint32_t* dev_err, cudaStream_t st);
cudaError_t launch_grouped_round(const GroupedShape& s, const float* dqacc, uint16_t* dq, cudaStream_t st);
cudaError_t launch_grouped_join(const GroupedShape& s, const float* part, int parts, uint16_t* dk, uint16_t* dv,
                                cudaStream_t st);

// map_stats: a TMA map over the bf16 statistics chunks (encode_stats_map);
// map_dq one over the fp32 dQ accumulator (encode_dq_map).  The accumulator must be zeroed unless
// attn_bwd_dq_stores_first(s).
cudaError_t launch_attn_bwd(const CUtensorMap& map_q, const CUtensorMap& map_k, const CUtensorMap& map_v,
                            const CUtensorMap& map_do, const CUtensorMap& map_stats, const CUtensorMap& map_dq,
                            const AttnShape& s, const uint16_t* k_raw, const float* rk, const float* gk, uint16_t* dk, uint16_t* dv,
                            float* dqacc, uint32_t* counters, float* dgk_part, uint32_t* dev_err, cudaStream_t st);
// Whether the first dQ contribution to each query tile is stored rather than
// added, so that the accumulator needs no zeroing: the deterministic mode in
// the [B, H, N, d] layout (one segment), whose 128-row tiles end at the
// tensor's end.
inline bool attn_bwd_dq_stores_first(const AttnShape& s) { return s.deterministic && s.seg.n == 1; }
// CTAs of the backward launch (one dgk partial each), and the counter words
// it needs zeroed (deterministic mode: one per query tile; else 0).
int attn_bwd_dgk_parts(const AttnShape& s);
int attn_bwd_counter_words(const AttnShape& s);

// --- QKV projection with the QK-RMSNorm epilogue ---------------------------
// Stream 0 is the image stream, stream 1 the caption stream; maps holds the
// TMA maps of x0, w0, x1, w1 (encode_rows_map: x; encode_heads_map: w, boxes of
// kQkvWRows rows).  A stream with M = 0 rows launches no tiles (its maps are
// then any valid map).
// Tiles: 256 rows x 256 columns by a pair of CTAs (qkv_uses_pairs), each
// loading half of the weight rows, or 128 rows x one head by one CTA.
constexpr int kQkvCols(int d, bool pair) { return pair ? 256 : d; }
constexpr int kQkvWRows(int d, bool pair) { return pair ? 128 : d; }
struct QkvLaunch {
  int H, C, N, d;
  bool pair;    // the tiles, as the weights' maps were made for (qkv_uses_pairs)
  int M[2];     // token rows B * N_s
  int N_s[2];   // tokens per batch item
  int row0[2];  // first row in the joint sequence
  const float* bias[2];  // [3 H d] fp32 or null
  bool e4m3;             // 8-bit tokens and weights, with the scales of their rows:
  const float *sx[2], *sw[2];
  const float *gq, *gk;
  uint16_t* out[3];  // q, k, v
  uint16_t* hat[2];  // q_hat, k_hat
  bool wide;         // those five at 32-byte boundaries
  float* r[2];       // rq, rk
};
// Low-rank adapters of the batch items beside the projection (bf16 only).
struct LoraLaunch {
  int n_adapters, rank;
  const int* index;    // [B] the items' adapters
  const float* scale;  // [n_adapters]
  bool on[2];          // whether a stream has adapters (and rows)
  uint16_t* u[2];      // scratch [M, 3 ceil(rank / 16), 3, 16]
};
// lora_maps (with lora): encode_u_map maps of both streams' U, then
// encode_up_map maps of their up weights (boxes of kQkvWRows rows); a stream
// without adapters: any valid map.
cudaError_t launch_qkv_norm(const CUtensorMap (&maps)[4], const QkvLaunch& a,
                            uint32_t* dev_err, cudaStream_t st, const LoraLaunch* lora = nullptr,
                            const CUtensorMap* lora_maps = nullptr);
bool qkv_uses_pairs(const QkvLaunch& a);
cudaError_t launch_qkv_norm_e4m3(const CUtensorMap (&maps)[4], const QkvLaunch& a,
                                 uint32_t* dev_err, cudaStream_t st);
cudaError_t launch_qkv_norm_lora(const CUtensorMap (&maps)[4], const QkvLaunch& a,
                                 uint32_t* dev_err, cudaStream_t st, const LoraLaunch* lora,
                                 const CUtensorMap* lora_maps);
// U = scale X A^T in three bf16 terms, before launch_qkv_norm.  x: [B, N_s, C] as
// encode_bhnd_map maps; down: the adapters' [3 n, rank, C] as
// encode_bhnd_map_rows(..., 16 ceil(rank / 16)) maps.
cudaError_t launch_lora_down(const CUtensorMap (&x)[2], const CUtensorMap (&down)[2], const LoraLaunch& l,
                             const QkvLaunch& a, int B, uint32_t* dev_err, cudaStream_t st);
// A 2-D TMA map over a row-major [rows, cols] matrix of bf16 (or, with e4m3,
// 8-bit) values with a (128 bytes, 128) box and 128-byte swizzle (a row's bytes
// a multiple of 16).
bool encode_rows_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, bool e4m3);
// The projection's order of columns: a box row 64 g + 4 j + b is matrix row 64 g
// + 16 b + j, so that four lanes that read one row of the accumulator four
// columns at a time end with 16 consecutive columns each.
// Weights [rows, cols], rows a multiple of 64, in that order: a 4-D map
// (cols, b, j, g) with box_rows (a multiple of 64) rows a box, otherwise as above.
bool encode_heads_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int box_rows, bool e4m3);
// U [rows, units, 3, 16]: a 3-D map (16, rows, 3 units), the three terms of 16
// columns of 128 rows a box, term by term, 32-byte swizzle.
bool encode_u_map(CUtensorMap* map, const uint16_t* u, int64_t rows, int units);
// n adapters' up weights [rows, rank] in that order: a 5-D map (rank, b, j, g,
// adapter), 16 of the rank and box_rows rows a box, 32-byte swizzle.
bool encode_up_map(CUtensorMap* map, const uint16_t* up, int n, int64_t rows, int rank, int box_rows);

// Encodes a 3-D TMA map over a [BH, N, d] bf16 tensor with a (64, 128, 1)
// box and 128-byte swizzle.  Returns false if the driver rejects it.
bool encode_bhnd_map(CUtensorMap* map, const void* base, int BH, int N, int d);
// The same with a (64, box_rows, 1) box.
bool encode_bhnd_map_rows(CUtensorMap* map, const void* base, int BH, int N, int d, int box_rows);
// A 3-D TMA map over [BH, prows, 16] bf16 statistics chunks with a
// (16, 128, 1) box and 32-byte swizzle.
bool encode_stats_map(CUtensorMap* map, const void* base, int BH, int prows);
// A 3-D TMA map over a [BH, rows, 64] fp32 accumulator with a (32, 128, 1)
// box and 128-byte swizzle.
bool encode_dq_map(CUtensorMap* map, const void* base, int BH, int rows, int d);

}  // namespace jattn
