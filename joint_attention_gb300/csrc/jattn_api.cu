// jattn_api.cu — the C ABI of libjattn (declared in include/jattn.h):
// argument validation, per-call scratch, TMA tensor maps and the launch
// sequence of the forward and backward passes.
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "jattn.h"
#include "jattn_internal.h"
#include "sm103_ptx.cuh"

namespace jattn {
namespace {

constexpr int kVersion = 100;  // 0.1.0
constexpr int kMaxDevices = 64;

// Device error word written by the kernels' bounded waits (one per device).
__device__ uint32_t g_dev_err;

// Backward mode set by jattn_set_deterministic (applies to later calls).
std::atomic<int> g_deterministic{0};

// Text of the last failure seen by an entry point on this thread.
thread_local char g_last_msg[256] = "no error";

int fail(int status, const char* where, cudaError_t e = cudaSuccess) {
  if (e != cudaSuccess)
    snprintf(g_last_msg, sizeof(g_last_msg), "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
  else
    snprintf(g_last_msg, sizeof(g_last_msg), "%s", where);
  return status;
}

uint32_t* dev_err_ptr() {
  static uint32_t* ptrs[kMaxDevices] = {nullptr};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!ptrs[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_dev_err) != cudaSuccess) return nullptr;
    ptrs[dev] = static_cast<uint32_t*>(p);
  }
  return ptrs[dev];
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// ---------------------------------------------------------------------------
// Kernel timing: CUDA event pairs around each launch while enabled.
// ---------------------------------------------------------------------------
struct Prof {
  std::mutex mu;
  bool on = false;
  struct Rec {
    int kind;
    cudaEvent_t a, b;
  };
  std::vector<Rec> pending;
  std::vector<cudaEvent_t> pool;
  long long launches[JATTN_TOKEN_KERNEL_END] = {0};  // by kind (both ranges of kinds)
  double ms[JATTN_TOKEN_KERNEL_END] = {0};

  cudaEvent_t get() {
    if (!pool.empty()) {
      cudaEvent_t e = pool.back();
      pool.pop_back();
      return e;
    }
    cudaEvent_t e = nullptr;
    if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
    return e;
  }
};
Prof& prof() {
  static Prof p;
  return p;
}

// Brackets one launch; a no-op unless timing is enabled.
class Timed {
 public:
  Timed(int kind, cudaStream_t st) : kind_(kind), st_(st) {
    Prof& p = prof();
    std::lock_guard<std::mutex> lock(p.mu);
    if (!p.on) return;
    a_ = p.get();
    b_ = p.get();
    if (a_ && b_) cudaEventRecord(a_, st_);
  }
  ~Timed() {
    if (!a_ || !b_) return;
    cudaEventRecord(b_, st_);
    Prof& p = prof();
    std::lock_guard<std::mutex> lock(p.mu);
    p.pending.push_back({kind_, a_, b_});
  }

 private:
  int kind_;
  cudaStream_t st_;
  cudaEvent_t a_ = nullptr, b_ = nullptr;
};

struct Range {
  uintptr_t lo, hi;
};
bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
Range range_of(const void* p, size_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + bytes};
}
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Shape {
  int B, H, N, d, BH;  // BH heads of N rows each (packed variable-length: H heads of T rows)
  size_t rows;         // BH * N
  size_t elems;        // BH * N * d
  SegTable seg;        // the heads' segments
};

int check_shape(int B, int H, int N_img, int N_txt, int d, Shape* s) {
  if (B <= 0 || H <= 0 || d <= 0 || N_img < 0 || N_txt < 0) return JATTN_ERR_INVALID_ARG;
  const int64_t N = static_cast<int64_t>(N_img) + N_txt;
  if (N < 1) return JATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return JATTN_ERR_UNSUPPORTED;
  const int64_t BH = static_cast<int64_t>(B) * H;
  if (BH > 65535) return JATTN_ERR_INVALID_ARG;  // grid y extent
  const int64_t elems = BH * N * d;
  if (elems >= (int64_t{1} << 31)) return JATTN_ERR_INVALID_ARG;
  s->B = B;
  s->H = H;
  s->N = static_cast<int>(N);
  s->d = d;
  s->BH = static_cast<int>(BH);
  s->rows = static_cast<size_t>(BH * N);
  s->elems = static_cast<size_t>(elems);
  make_uniform_seg_table(&s->seg, s->N);
  return JATTN_OK;
}

// Packed variable-length layout: H heads of T = cu[n] rows, one segment per
// sequence.  cu is a host array of n + 1 row offsets.
int check_shape_varlen(const int* cu, int n, int H, int d, Shape* s) {
  if (!cu || n < 1 || H <= 0 || d <= 0) return JATTN_ERR_INVALID_ARG;
  if (n > kMaxSegments) return JATTN_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return JATTN_ERR_UNSUPPORTED;
  if (H > 65535) return JATTN_ERR_INVALID_ARG;
  if (!make_seg_table(&s->seg, cu, n)) return JATTN_ERR_INVALID_ARG;
  const int64_t T = s->seg.rows;
  const int64_t elems = static_cast<int64_t>(H) * T * d;
  if (elems >= (int64_t{1} << 31) || static_cast<int64_t>(H) * s->seg.prows >= (int64_t{1} << 31))
    return JATTN_ERR_INVALID_ARG;
  s->B = 1;
  s->H = H;
  s->N = static_cast<int>(T);
  s->d = d;
  s->BH = H;
  s->rows = static_cast<size_t>(H) * T;
  s->elems = static_cast<size_t>(elems);
  return JATTN_OK;
}

// Bump allocator over one stream-ordered allocation.
struct Carve {
  uint8_t* base = nullptr;
  size_t off = 0;
  template <typename T>
  T* take(size_t count) {
    off = (off + 255) & ~static_cast<size_t>(255);
    T* p = reinterpret_cast<T*>(base + off);
    off += count * sizeof(T);
    return p;
  }
};

size_t fwd_scratch_bytes(const Shape& s) { return 2 * (s.elems * 2 + 256) + 256; }

// The activations a training forward keeps for its backward, at 256-byte
// aligned offsets of one caller buffer: q_hat, k_hat (bf16, q's shape), then
// 1/rms of every q and k row (fp32); then the backward's fp32 dQ accumulator
// (q's shape), which the forward zeroes with bandwidth it leaves idle, and the
// word that counts the forward CTAs that have zeroed their share.
struct SavedLayout {
  size_t qhat, khat, rq, rk, dq, zero_count, total;
};
SavedLayout saved_layout(const Shape& s) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  SavedLayout l;
  l.qhat = 0;
  l.khat = up(s.elems * 2);
  l.rq = l.khat + up(s.elems * 2);
  l.rk = l.rq + up(s.rows * 4);
  l.dq = l.rk + up(s.rows * 4);
  l.zero_count = l.dq + up(s.elems * 4);
  l.total = l.zero_count + 256;
  return l;
}

size_t bwd_scratch_bytes(const Shape& s, int nparts_q, int nparts_k, int counter_words, bool saved) {
  size_t b = 0;
  if (!saved) {
    b += 2 * (s.elems * 2 + 256);  // q_hat, k_hat
    b += 2 * (s.rows * 4 + 256);   // rq, rk
    b += s.elems * 4 + 256;        // dq accumulator
  }
  b += static_cast<size_t>(s.BH) * s.seg.prows * 32 + 256;  // statistics chunks
  b += (static_cast<size_t>(nparts_q) + nparts_k) * s.d * 4 + 512; // dg partials
  b += 4 * (1 + static_cast<size_t>(counter_words)) + 256;      // dg ticket, dQ order counters
  return b + 256;
}

}  // namespace

bool make_seg_table(SegTable* t, const int* cu, int n) {
  if (!t || !cu || n < 1 || n > kMaxSegments || cu[0] != 0) return false;
  t->n = n;
  t->cu[0] = 0;
  t->pcu[0] = 0;
  for (int i = 0; i < n; ++i) {
    if (cu[i + 1] <= cu[i]) return false;  // every segment has a row
    const int64_t padded = t->pcu[i] + (static_cast<int64_t>(cu[i + 1] - cu[i]) + 127) / 128 * 128;
    if (padded >= (int64_t{1} << 31)) return false;
    t->cu[i + 1] = cu[i + 1];
    t->pcu[i + 1] = static_cast<int>(padded);
  }
  t->rows = cu[n];
  t->prows = t->pcu[n];
  return true;
}

void make_uniform_seg_table(SegTable* t, int N) {
  const int cu[2] = {0, N};
  make_seg_table(t, cu, 1);
}

bool encode_bhnd_map(CUtensorMap* map, const void* base, int BH, int N, int d) {
  return encode_bhnd_map_rows(map, base, BH, N, d, 128);
}

bool encode_bhnd_map_rows(CUtensorMap* map, const void* base, int BH, int N, int d, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(N) * d * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool encode_rows_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, bool e4m3) {
  auto fn = encode_fn();
  if (!fn) return false;
  const int size = e4m3 ? 1 : 2;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * size};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / size), 128};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                  const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool encode_heads_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int box_rows, bool e4m3) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t size = e4m3 ? 1 : 2, row = static_cast<cuuint64_t>(cols) * size;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(cols), 4, 16, static_cast<cuuint64_t>(rows) / 64};
  cuuint64_t strides[3] = {16 * row, row, 64 * row};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(128 / size), 4, 16, static_cast<cuuint32_t>(box_rows) / 64};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = fn(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                  const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool encode_u_map(CUtensorMap* map, const uint16_t* u, int64_t rows, int units) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {16, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(3 * units)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(units) * 96, 32};
  cuuint32_t box[3] = {16, 128, 3};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(u), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool encode_up_map(CUtensorMap* map, const uint16_t* up, int n, int64_t rows, int rank, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(rank) * 2;
  cuuint64_t dims[5] = {static_cast<cuuint64_t>(rank), 4, 16, static_cast<cuuint64_t>(rows) / 64,
                        static_cast<cuuint64_t>(n)};
  cuuint64_t strides[4] = {16 * row, row, 64 * row, static_cast<cuuint64_t>(rows) * row};
  cuuint32_t box[5] = {16, 4, 16, static_cast<cuuint32_t>(box_rows) / 64, 1};
  cuuint32_t es[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<uint16_t*>(up), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_32B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool encode_dq_map(CUtensorMap* map, const void* base, int BH, int rows, int d) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 4, static_cast<cuuint64_t>(rows) * d * 4};
  cuuint32_t box[3] = {32, 128, 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool encode_stats_map(CUtensorMap* map, const void* base, int BH, int prows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {16, static_cast<cuuint64_t>(prows), static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {32, static_cast<cuuint64_t>(prows) * 32};
  cuuint32_t box[3] = {16, 128, 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace jattn

using namespace jattn;

namespace jattn {
namespace {

// The fixed scratch of jattn_fwd_noalloc (see include/jattn.h): one array per
// device, looked up once per device and then shared by every call.
static __device__ __align__(256) uint8_t g_noalloc_scratch[JATTN_NOALLOC_SCRATCH_BYTES];

uint8_t* noalloc_scratch_ptr() {
  static uint8_t* ptrs[kMaxDevices] = {nullptr};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!ptrs[dev]) {
    void* p = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
    if (e != cudaSuccess) {
      fail(JATTN_ERR_CUDA, "cudaGetSymbolAddress(no-alloc scratch)", e);
      return nullptr;
    }
    ptrs[dev] = static_cast<uint8_t*>(p);
  }
  return ptrs[dev];
}

}  // namespace
}  // namespace jattn

extern "C" int jattn_fwd_noalloc(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq,
                                 const float* gk, int B, int H, int N_img, int N_txt, int d, jattn_bf16* out,
                                 float* lse, void* stream) {
  if (!q || !k || !v || !gq || !gk || !out || !lse) return JATTN_ERR_INVALID_ARG;
  Shape s;
  int rc = check_shape(B, H, N_img, N_txt, d, &s);
  if (rc != JATTN_OK) return rc;
  const void* ptrs[] = {q, k, v, gq, gk, out, lse};
  for (const void* p : ptrs)
    if (!aligned16(p)) return JATTN_ERR_MISALIGNED;
  const size_t tb = s.elems * 2;
  const Range ins[] = {range_of(q, tb), range_of(k, tb), range_of(v, tb), range_of(gq, s.d * 4),
                       range_of(gk, s.d * 4)};
  const Range outs[] = {range_of(out, tb), range_of(lse, s.rows * 4)};
  for (const Range& o : outs)
    for (const Range& i : ins)
      if (overlaps(o, i)) return JATTN_ERR_ALIAS;
  if (overlaps(outs[0], outs[1])) return JATTN_ERR_ALIAS;
  const size_t part = (tb + 255) & ~static_cast<size_t>(255);
  if (2 * part > JATTN_NOALLOC_SCRATCH_BYTES) return JATTN_ERR_SCRATCH_LIMIT;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t* err = dev_err_ptr();
  if (!err) return fail(JATTN_ERR_CUDA, "device error word", cudaGetLastError());
  uint8_t* scratch = noalloc_scratch_ptr();
  if (!scratch) return JATTN_ERR_CUDA;
  uint16_t* qhat = reinterpret_cast<uint16_t*>(scratch);
  uint16_t* khat = reinterpret_cast<uint16_t*>(scratch + part);
  cudaError_t ce;
  {
    Timed t(JATTN_KERNEL_QK_NORM_FWD, st);
    ce = launch_qk_norm_fwd(q, k, gq, gk, qhat, khat, nullptr, nullptr, static_cast<int64_t>(s.rows), s.d, err, st);
  }
  if (ce != cudaSuccess) return fail(JATTN_ERR_CUDA, "qk_norm_fwd launch", ce);
  CUtensorMap mq, mk, mv;
  if (!encode_bhnd_map(&mq, qhat, s.BH, s.N, s.d) || !encode_bhnd_map(&mk, khat, s.BH, s.N, s.d) ||
      !encode_bhnd_map(&mv, v, s.BH, s.N, s.d))
    return fail(JATTN_ERR_CUDA, "cuTensorMapEncodeTiled");
  AttnShape as{s.BH, s.N, s.d, 1.0f / sqrtf(static_cast<float>(s.d)), s.seg};
  Timed t(JATTN_KERNEL_ATTN_FWD, st);
  ce = launch_attn_fwd(mq, mk, mv, as, out, lse, err, st);
  if (ce != cudaSuccess) return fail(JATTN_ERR_CUDA, "attn_fwd launch", ce);
  return JATTN_OK;
}

namespace {

// The forward for a validated shape (either layout); with `saved` non-null
// (a training forward) q_hat, k_hat and the rows' 1/rms go there instead of
// into scratch.
int fwd_body(const Shape& s, const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq,
             const float* gk, jattn_bf16* out, float* lse, void* saved, void* stream) {
  const void* ptrs[] = {q, k, v, gq, gk, out, lse, saved};
  for (const void* p : ptrs)
    if (!aligned16(p)) return JATTN_ERR_MISALIGNED;
  const size_t tb = s.elems * 2;
  const SavedLayout sl = saved_layout(s);
  const Range ins[] = {range_of(q, tb), range_of(k, tb), range_of(v, tb), range_of(gq, s.d * 4),
                       range_of(gk, s.d * 4)};
  const Range outs[] = {range_of(out, tb), range_of(lse, s.rows * 4), range_of(saved, saved ? sl.total : 0)};
  for (size_t a = 0; a < sizeof(outs) / sizeof(outs[0]); ++a) {
    for (const Range& i : ins)
      if (overlaps(outs[a], i)) return JATTN_ERR_ALIAS;
    for (size_t b = a + 1; b < sizeof(outs) / sizeof(outs[0]); ++b)
      if (overlaps(outs[a], outs[b])) return JATTN_ERR_ALIAS;
  }

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t* err = dev_err_ptr();
  if (!err) return fail(JATTN_ERR_CUDA, "device error word", cudaGetLastError());
  Carve cv;
  uint16_t *qhat, *khat;
  float *rq = nullptr, *rk = nullptr;
  cudaError_t ce;
  if (saved) {
    uint8_t* base = static_cast<uint8_t*>(saved);
    qhat = reinterpret_cast<uint16_t*>(base + sl.qhat);
    khat = reinterpret_cast<uint16_t*>(base + sl.khat);
    rq = reinterpret_cast<float*>(base + sl.rq);
    rk = reinterpret_cast<float*>(base + sl.rk);
  } else {
    ce = cudaMallocAsync(reinterpret_cast<void**>(&cv.base), fwd_scratch_bytes(s), st);
    if (ce != cudaSuccess) return fail(JATTN_ERR_CUDA, "cudaMallocAsync", ce);
    qhat = cv.take<uint16_t>(s.elems);
    khat = cv.take<uint16_t>(s.elems);
  }
  int status = JATTN_OK;
  CUtensorMap mq, mk, mv;
  {
    Timed t(JATTN_KERNEL_QK_NORM_FWD, st);
    ce = launch_qk_norm_fwd(q, k, gq, gk, qhat, khat, rq, rk, static_cast<int64_t>(s.rows), s.d, err, st);
  }
  if (ce != cudaSuccess) {
    status = fail(JATTN_ERR_CUDA, "qk_norm_fwd launch", ce);
  } else if (!encode_bhnd_map(&mq, qhat, s.BH, s.N, s.d) || !encode_bhnd_map(&mk, khat, s.BH, s.N, s.d) ||
             !encode_bhnd_map(&mv, v, s.BH, s.N, s.d)) {
    status = fail(JATTN_ERR_CUDA, "cuTensorMapEncodeTiled");
  } else {
    AttnShape as{s.BH, s.N, s.d, 1.0f / sqrtf(static_cast<float>(s.d)), s.seg};
    Timed t(JATTN_KERNEL_ATTN_FWD, st);
    uint8_t* base = static_cast<uint8_t*>(saved);
    ce = launch_attn_fwd(mq, mk, mv, as, out, lse, err, st, saved ? reinterpret_cast<float*>(base + sl.dq) : nullptr,
                         saved ? reinterpret_cast<uint32_t*>(base + sl.zero_count) : nullptr);
    if (ce != cudaSuccess) status = fail(JATTN_ERR_CUDA, "attn_fwd launch", ce);
  }
  if (cv.base) {
    ce = cudaFreeAsync(cv.base, st);
    if (ce != cudaSuccess) status = fail(JATTN_ERR_CUDA, "cudaFreeAsync", ce);
  }
  return status;
}

}  // namespace

extern "C" int jattn_fwd(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq,
                         const float* gk, int B, int H, int N_img, int N_txt, int d, jattn_bf16* out, float* lse,
                         void* stream) {
  if (!q || !k || !v || !gq || !gk || !out || !lse) return JATTN_ERR_INVALID_ARG;
  Shape s;
  int rc = check_shape(B, H, N_img, N_txt, d, &s);
  if (rc != JATTN_OK) return rc;
  return fwd_body(s, q, k, v, gq, gk, out, lse, nullptr, stream);
}

extern "C" int jattn_fwd_varlen(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq,
                                const float* gk, const int* cu_seqlens, int n_seqs, int H, int d, jattn_bf16* out,
                                float* lse, void* stream) {
  if (!q || !k || !v || !gq || !gk || !out || !lse) return JATTN_ERR_INVALID_ARG;
  Shape s;
  int rc = check_shape_varlen(cu_seqlens, n_seqs, H, d, &s);
  if (rc != JATTN_OK) return rc;
  return fwd_body(s, q, k, v, gq, gk, out, lse, nullptr, stream);
}

namespace {

// The backward for a validated shape (either layout); with `saved` non-null
// q_hat, k_hat and the rows' 1/rms come from a training forward instead of
// being recomputed.
int bwd_body(const Shape& s, const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq,
             const float* gk, const jattn_bf16* out, const float* lse, const jattn_bf16* dout, void* saved,
             jattn_bf16* dq, jattn_bf16* dk, jattn_bf16* dv, float* dgq, float* dgk, void* stream) {
  const void* ptrs[] = {q, k, v, gq, gk, out, lse, dout, saved, dq, dk, dv, dgq, dgk};
  for (const void* p : ptrs)
    if (!aligned16(p)) return JATTN_ERR_MISALIGNED;
  const size_t tb = s.elems * 2;
  const size_t gb = static_cast<size_t>(s.d) * 4;
  const SavedLayout sl = saved_layout(s);
  const Range ins[] = {range_of(q, tb),  range_of(k, tb),   range_of(v, tb),           range_of(gq, gb),
                       range_of(gk, gb), range_of(out, tb), range_of(lse, s.rows * 4), range_of(dout, tb),
                       range_of(saved, saved ? sl.total : 0)};
  const Range outs[] = {range_of(dq, tb), range_of(dk, tb), range_of(dv, tb), range_of(dgq, gb), range_of(dgk, gb)};
  for (size_t a = 0; a < sizeof(outs) / sizeof(outs[0]); ++a) {
    for (const Range& i : ins)
      if (overlaps(outs[a], i)) return JATTN_ERR_ALIAS;
    for (size_t b = a + 1; b < sizeof(outs) / sizeof(outs[0]); ++b)
      if (overlaps(outs[a], outs[b])) return JATTN_ERR_ALIAS;
  }

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t* err = dev_err_ptr();
  if (!err) return fail(JATTN_ERR_CUDA, "device error word", cudaGetLastError());
  AttnShape as{s.BH, s.N, s.d, 1.0f / sqrtf(static_cast<float>(s.d)), s.seg};
  const int nparts_q = q_norm_bwd_parts(s.d);
  as.deterministic = g_deterministic.load(std::memory_order_relaxed) != 0;
  const int nparts_k = attn_bwd_dgk_parts(as);
  const int counter_words = attn_bwd_counter_words(as);
  Carve cv;
  cudaError_t ce = cudaMallocAsync(reinterpret_cast<void**>(&cv.base),
                                   bwd_scratch_bytes(s, nparts_q, nparts_k, counter_words, saved != nullptr), st);
  if (ce != cudaSuccess) return fail(JATTN_ERR_CUDA, "cudaMallocAsync", ce);
  uint16_t *qhat, *khat;
  float *rq, *rk, *dqacc;
  uint32_t* zero_count = nullptr;
  if (saved) {
    uint8_t* base = static_cast<uint8_t*>(saved);
    qhat = reinterpret_cast<uint16_t*>(base + sl.qhat);
    khat = reinterpret_cast<uint16_t*>(base + sl.khat);
    rq = reinterpret_cast<float*>(base + sl.rq);
    rk = reinterpret_cast<float*>(base + sl.rk);
    dqacc = reinterpret_cast<float*>(base + sl.dq);
    zero_count = reinterpret_cast<uint32_t*>(base + sl.zero_count);
  } else {
    qhat = cv.take<uint16_t>(s.elems);
    khat = cv.take<uint16_t>(s.elems);
    rq = cv.take<float>(s.rows);
    rk = cv.take<float>(s.rows);
    dqacc = cv.take<float>(s.elems);
  }
  uint16_t* stats = cv.take<uint16_t>(static_cast<size_t>(s.BH) * s.seg.prows * 16);
  float* dgq_part = cv.take<float>(static_cast<size_t>(nparts_q) * s.d);
  float* dgk_part = cv.take<float>(static_cast<size_t>(nparts_k) * s.d);
  // The gain-gradient ticket, then (deterministic mode) one dQ order counter
  // per query tile; the preparation zeroes them all.
  unsigned int* dg_ticket = cv.take<unsigned int>(1 + static_cast<size_t>(counter_words));

  int status = JATTN_OK;
  CUtensorMap mq, mk, mv, mdo, mstats, mdqacc;
  {
    Timed t(JATTN_KERNEL_BWD_PREP, st);
    // Saved activations: the preparation computes only the statistics.
    ce = launch_bwd_prep(q, k, gq, gk, out, dout, lse, saved ? nullptr : qhat, khat, rq, rk, stats,
                         sqrtf(static_cast<float>(s.d)), attn_bwd_dq_stores_first(as) ? nullptr : dqacc, dg_ticket,
                         1 + counter_words, s.BH, s.seg, s.d, err, st, zero_count,
                         static_cast<uint32_t>(attn_fwd_grid(as)));
  }
  if (ce != cudaSuccess) {
    status = fail(JATTN_ERR_CUDA, "bwd_prep launch", ce);
  } else if (!encode_bhnd_map(&mq, qhat, s.BH, s.N, s.d) || !encode_bhnd_map(&mk, khat, s.BH, s.N, s.d) ||
             !encode_bhnd_map(&mv, v, s.BH, s.N, s.d) || !encode_bhnd_map(&mdo, dout, s.BH, s.N, s.d) ||
             !encode_stats_map(&mstats, stats, s.BH, s.seg.prows) ||
             !encode_dq_map(&mdqacc, dqacc, s.BH, s.seg.rows, s.d)) {
    status = fail(JATTN_ERR_CUDA, "cuTensorMapEncodeTiled");
  } else {
    const char* stage = "attn_bwd launch";
    {
      Timed t(JATTN_KERNEL_ATTN_BWD, st);
      ce = launch_attn_bwd(mq, mk, mv, mdo, mstats, mdqacc, as, k, rk, gk, dk, dv, dqacc, dg_ticket + 1, dgk_part, err,
                           st);
    }
    if (ce == cudaSuccess) {
      stage = "q_norm_bwd launch";
      Timed t(JATTN_KERNEL_Q_NORM_BWD, st);
      ce = launch_q_norm_bwd(dqacc, q, rq, gq, as.scale, dq, dgq_part, nparts_q, static_cast<int64_t>(s.rows),
                             dgk_part, nparts_k, dg_ticket, dgq, dgk, s.d, err, st, zero_count);
    }
    if (ce != cudaSuccess) status = fail(JATTN_ERR_CUDA, stage, ce);
  }
  ce = cudaFreeAsync(cv.base, st);
  if (ce != cudaSuccess) status = fail(JATTN_ERR_CUDA, "cudaFreeAsync", ce);
  return status;
}

}  // namespace

extern "C" int jattn_bwd(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq,
                         const float* gk, const jattn_bf16* out, const float* lse, const jattn_bf16* dout,
                         jattn_bf16* dq, jattn_bf16* dk, jattn_bf16* dv, float* dgq, float* dgk, int B, int H,
                         int N_img, int N_txt, int d, void* stream) {
  if (!q || !k || !v || !gq || !gk || !out || !lse || !dout || !dq || !dk || !dv || !dgq || !dgk)
    return JATTN_ERR_INVALID_ARG;
  Shape s;
  int rc = check_shape(B, H, N_img, N_txt, d, &s);
  if (rc != JATTN_OK) return rc;
  return bwd_body(s, q, k, v, gq, gk, out, lse, dout, nullptr, dq, dk, dv, dgq, dgk, stream);
}

extern "C" int jattn_bwd_varlen(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq,
                                const float* gk, const jattn_bf16* out, const float* lse, const jattn_bf16* dout,
                                jattn_bf16* dq, jattn_bf16* dk, jattn_bf16* dv, float* dgq, float* dgk,
                                const int* cu_seqlens, int n_seqs, int H, int d, void* stream) {
  if (!q || !k || !v || !gq || !gk || !out || !lse || !dout || !dq || !dk || !dv || !dgq || !dgk)
    return JATTN_ERR_INVALID_ARG;
  Shape s;
  int rc = check_shape_varlen(cu_seqlens, n_seqs, H, d, &s);
  if (rc != JATTN_OK) return rc;
  return bwd_body(s, q, k, v, gq, gk, out, lse, dout, nullptr, dq, dk, dv, dgq, dgk, stream);
}

extern "C" size_t jattn_saved_bytes(int B, int H, int N_img, int N_txt, int d) {
  Shape s;
  if (check_shape(B, H, N_img, N_txt, d, &s) != JATTN_OK) return 0;
  return saved_layout(s).total;
}

extern "C" size_t jattn_saved_bytes_varlen(const int* cu_seqlens, int n_seqs, int H, int d) {
  Shape s;
  if (check_shape_varlen(cu_seqlens, n_seqs, H, d, &s) != JATTN_OK) return 0;
  return saved_layout(s).total;
}

extern "C" int jattn_fwd_train(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq,
                               const float* gk, int B, int H, int N_img, int N_txt, int d, jattn_bf16* out,
                               float* lse, void* saved, void* stream) {
  if (!q || !k || !v || !gq || !gk || !out || !lse || !saved) return JATTN_ERR_INVALID_ARG;
  Shape s;
  int rc = check_shape(B, H, N_img, N_txt, d, &s);
  if (rc != JATTN_OK) return rc;
  return fwd_body(s, q, k, v, gq, gk, out, lse, saved, stream);
}

extern "C" int jattn_fwd_train_varlen(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq,
                                      const float* gk, const int* cu_seqlens, int n_seqs, int H, int d,
                                      jattn_bf16* out, float* lse, void* saved, void* stream) {
  if (!q || !k || !v || !gq || !gk || !out || !lse || !saved) return JATTN_ERR_INVALID_ARG;
  Shape s;
  int rc = check_shape_varlen(cu_seqlens, n_seqs, H, d, &s);
  if (rc != JATTN_OK) return rc;
  return fwd_body(s, q, k, v, gq, gk, out, lse, saved, stream);
}

extern "C" int jattn_bwd_train(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v, const float* gq,
                               const float* gk, const jattn_bf16* out, const float* lse, const jattn_bf16* dout,
                               void* saved, jattn_bf16* dq, jattn_bf16* dk, jattn_bf16* dv, float* dgq,
                               float* dgk, int B, int H, int N_img, int N_txt, int d, void* stream) {
  if (!q || !k || !v || !gq || !gk || !out || !lse || !dout || !saved || !dq || !dk || !dv || !dgq || !dgk)
    return JATTN_ERR_INVALID_ARG;
  Shape s;
  int rc = check_shape(B, H, N_img, N_txt, d, &s);
  if (rc != JATTN_OK) return rc;
  return bwd_body(s, q, k, v, gq, gk, out, lse, dout, saved, dq, dk, dv, dgq, dgk, stream);
}

extern "C" int jattn_bwd_train_varlen(const jattn_bf16* q, const jattn_bf16* k, const jattn_bf16* v,
                                      const float* gq, const float* gk, const jattn_bf16* out, const float* lse,
                                      const jattn_bf16* dout, void* saved, jattn_bf16* dq, jattn_bf16* dk,
                                      jattn_bf16* dv, float* dgq, float* dgk, const int* cu_seqlens, int n_seqs,
                                      int H, int d, void* stream) {
  if (!q || !k || !v || !gq || !gk || !out || !lse || !dout || !saved || !dq || !dk || !dv || !dgq || !dgk)
    return JATTN_ERR_INVALID_ARG;
  Shape s;
  int rc = check_shape_varlen(cu_seqlens, n_seqs, H, d, &s);
  if (rc != JATTN_OK) return rc;
  return bwd_body(s, q, k, v, gq, gk, out, lse, dout, saved, dq, dk, dv, dgq, dgk, stream);
}

namespace {

// One projection call: the image (0) and caption (1) streams' operands, and
// what the 8-bit or the adapter form adds.
struct QkvCall {
  const void* x[2];
  const void* w[2];
  const float* bias[2];
  const float *gq, *gk;
  int B, H, N_img, N_txt, d, C;
  jattn_bf16 *q, *k, *v;
  void* saved;
  void* stream;
  bool e4m3 = false;
  const float* sx[2] = {nullptr, nullptr};
  const float* sw[2] = {nullptr, nullptr};
  bool lora = false;
  const jattn_bf16* down[2] = {nullptr, nullptr};
  const jattn_bf16* up[2] = {nullptr, nullptr};
  const float* scale = nullptr;
  const int* index = nullptr;
  int n_adapters = 0, rank = 0;
  void* work = nullptr;
};

size_t lora_u_bytes(int64_t rows, int rank) {
  const int64_t r16 = (rank + 15) / 16 * 16;
  return (static_cast<size_t>(rows) * 3 * 3 * r16 * 2 + 255) & ~static_cast<size_t>(255);
}

int check_lora(int rank) {
  if (rank <= 0) return JATTN_ERR_INVALID_ARG;
  return rank % 8 != 0 || rank > JATTN_MAX_RANK ? JATTN_ERR_UNSUPPORTED : JATTN_OK;
}

int qkv_body(const QkvCall& c) {
  const int n_s[2] = {c.N_img, c.N_txt};
  if (!c.gq || !c.gk || !c.q || !c.k || !c.v || !c.saved) return JATTN_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i) {
    if (n_s[i] > 0 && (!c.x[i] || !c.w[i])) return JATTN_ERR_INVALID_ARG;
    if (c.e4m3 && n_s[i] > 0 && (!c.sx[i] || !c.sw[i])) return JATTN_ERR_INVALID_ARG;
    if ((c.down[i] == nullptr) != (c.up[i] == nullptr)) return JATTN_ERR_INVALID_ARG;
  }
  if (c.lora && (!c.scale || !c.index || !c.work || c.n_adapters <= 0)) return JATTN_ERR_INVALID_ARG;
  Shape s;
  int rc = check_shape(c.B, c.H, c.N_img, c.N_txt, c.d, &s);
  if (rc != JATTN_OK) return rc;
  const int d = c.d, C = c.C;
  if (C <= 0) return JATTN_ERR_INVALID_ARG;
  // TMA row stride: a multiple of 16 bytes.
  const int size = c.e4m3 ? 1 : 2;
  if (C * static_cast<int64_t>(size) % 16 != 0) return JATTN_ERR_UNSUPPORTED;
  if (c.lora && (rc = check_lora(c.rank)) != JATTN_OK) return rc;
  const int64_t ycols = 3 * static_cast<int64_t>(c.H) * d;
  const int64_t limit = int64_t{1} << 31;
  if (ycols * C >= limit || static_cast<int64_t>(c.B) * c.N_img * C >= limit ||
      static_cast<int64_t>(c.B) * c.N_txt * C >= limit)
    return JATTN_ERR_INVALID_ARG;
  if (c.lora && (3 * static_cast<int64_t>(c.n_adapters) >= limit)) return JATTN_ERR_INVALID_ARG;
  const void* ptrs[] = {c.x[0], c.w[0],  c.bias[0], c.x[1],    c.w[1],    c.bias[1], c.gq,      c.gk,
                        c.q,    c.k,     c.v,       c.saved,   c.sx[0],   c.sx[1],   c.sw[0],   c.sw[1],
                        c.scale, c.index, c.work,   c.down[0], c.down[1], c.up[0],   c.up[1]};
  for (const void* p : ptrs)
    if (!aligned16(p)) return JATTN_ERR_MISALIGNED;
  const size_t tb = s.elems * 2;
  const SavedLayout sl = saved_layout(s);
  const size_t wb = static_cast<size_t>(ycols) * C * size, bb = static_cast<size_t>(ycols) * 4;
  auto bytes_if = [](bool on, size_t b) { return on ? b : size_t{0}; };
  Range ins[20];
  int n_in = 0;
  for (int i = 0; i < 2; ++i) {
    const bool on = n_s[i] > 0;
    const size_t rows = static_cast<size_t>(c.B) * n_s[i], n = static_cast<size_t>(c.n_adapters);
    ins[n_in++] = range_of(c.x[i], rows * C * size);
    ins[n_in++] = range_of(c.w[i], bytes_if(on, wb));
    ins[n_in++] = range_of(c.bias[i], bytes_if(on && c.bias[i], bb));
    ins[n_in++] = range_of(c.sx[i], bytes_if(c.sx[i], rows * 4));
    ins[n_in++] = range_of(c.sw[i], bytes_if(on && c.sw[i], bb));
    ins[n_in++] = range_of(c.down[i], bytes_if(on && c.down[i], n * 3 * c.rank * C * 2));
    ins[n_in++] = range_of(c.up[i], bytes_if(on && c.up[i], n * ycols * c.rank * 2));
  }
  ins[n_in++] = range_of(c.gq, d * 4);
  ins[n_in++] = range_of(c.gk, d * 4);
  ins[n_in++] = range_of(c.scale, bytes_if(c.lora, static_cast<size_t>(c.n_adapters) * 4));
  ins[n_in++] = range_of(c.index, bytes_if(c.lora, static_cast<size_t>(c.B) * 4));
  const size_t u_img = c.lora ? lora_u_bytes(static_cast<int64_t>(c.B) * c.N_img, c.rank) : 0;
  const size_t u_txt = c.lora ? lora_u_bytes(static_cast<int64_t>(c.B) * c.N_txt, c.rank) : 0;
  const Range outs[] = {range_of(c.q, tb), range_of(c.k, tb), range_of(c.v, tb), range_of(c.saved, sl.total),
                        range_of(c.work, u_img + u_txt)};
  for (size_t a = 0; a < sizeof(outs) / sizeof(outs[0]); ++a) {
    for (int i = 0; i < n_in; ++i)
      if (overlaps(outs[a], ins[i])) return JATTN_ERR_ALIAS;
    for (size_t b = a + 1; b < sizeof(outs) / sizeof(outs[0]); ++b)
      if (overlaps(outs[a], outs[b])) return JATTN_ERR_ALIAS;
  }

  cudaStream_t st = static_cast<cudaStream_t>(c.stream);
  uint32_t* err = dev_err_ptr();
  if (!err) return fail(JATTN_ERR_CUDA, "device error word", cudaGetLastError());
  uint8_t* base = static_cast<uint8_t*>(c.saved);
  QkvLaunch a;
  a.H = c.H;
  a.C = C;
  a.N = s.N;
  a.d = d;
  a.e4m3 = c.e4m3;
  // Stream 0: the image rows (after the caption rows); stream 1: the caption rows.
  for (int i = 0; i < 2; ++i) {
    a.M[i] = c.B * n_s[i];
    a.N_s[i] = n_s[i];
    a.row0[i] = i == 0 ? c.N_txt : 0;
    a.bias[i] = c.bias[i];
    a.sx[i] = c.sx[i];
    a.sw[i] = c.sw[i];
  }
  a.gq = c.gq;
  a.gk = c.gk;
  a.out[0] = c.q;
  a.out[1] = c.k;
  a.out[2] = c.v;
  a.hat[0] = reinterpret_cast<uint16_t*>(base + sl.qhat);
  a.hat[1] = reinterpret_cast<uint16_t*>(base + sl.khat);
  a.r[0] = reinterpret_cast<float*>(base + sl.rq);
  a.r[1] = reinterpret_cast<float*>(base + sl.rk);
  a.wide = true;
  for (const void* o : {a.out[0], a.out[1], a.out[2], a.hat[0], a.hat[1]})
    a.wide = a.wide && reinterpret_cast<uintptr_t>(o) % 32 == 0;
  a.pair = qkv_uses_pairs(a);
  const int w_rows = kQkvWRows(d, a.pair);
  CUtensorMap maps[4];
  for (int i = 0; i < 2; ++i) {
    const int j = n_s[i] ? i : 1 - i;  // a stream without rows launches no tiles: any valid map
    if (!encode_rows_map(&maps[2 * i], c.x[j], a.M[j], C, c.e4m3) ||
        !encode_heads_map(&maps[2 * i + 1], c.w[j], ycols, C, w_rows, c.e4m3))
      return fail(JATTN_ERR_CUDA, "cuTensorMapEncodeTiled");
  }
  cudaError_t ce;
  LoraLaunch l;
  CUtensorMap lora_maps[4], down_maps[2], item_maps[2];
  if (c.lora) {
    l.n_adapters = c.n_adapters;
    l.rank = c.rank;
    l.index = c.index;
    l.scale = c.scale;
    l.u[0] = static_cast<uint16_t*>(c.work);
    l.u[1] = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(c.work) + u_img);
    const int r16 = (c.rank + 15) / 16 * 16;
    for (int i = 0; i < 2; ++i) {
      l.on[i] = c.down[i] && n_s[i] > 0;
      if (!l.on[i]) {
        lora_maps[i] = lora_maps[2 + i] = down_maps[i] = item_maps[i] = maps[0];
      } else if (!encode_u_map(&lora_maps[i], l.u[i], a.M[i], 3 * r16 / 16) ||
                 !encode_up_map(&lora_maps[2 + i], c.up[i], c.n_adapters, ycols, c.rank, w_rows) ||
                 !encode_bhnd_map_rows(&down_maps[i], c.down[i], 3 * c.n_adapters, c.rank, C, r16) ||
                 !encode_bhnd_map(&item_maps[i], c.x[i], c.B, n_s[i], C)) {
        return fail(JATTN_ERR_CUDA, "cuTensorMapEncodeTiled");
      }
    }
    {
      Timed t(JATTN_KERNEL_LORA_DOWN, st);
      ce = launch_lora_down(item_maps, down_maps, l, a, c.B, err, st);
    }
    if (ce != cudaSuccess) return fail(JATTN_ERR_CUDA, "lora_down launch", ce);
  }
  {
    Timed t(JATTN_KERNEL_QKV_NORM, st);
    ce = launch_qkv_norm(maps, a, err, st, c.lora ? &l : nullptr, lora_maps);
  }
  if (ce != cudaSuccess) return fail(JATTN_ERR_CUDA, "qkv_norm launch", ce);
  return JATTN_OK;
}

}  // namespace

extern "C" int jattn_qkv_norm(const jattn_bf16* x_img, const jattn_bf16* w_img, const float* b_img,
                              const jattn_bf16* x_txt, const jattn_bf16* w_txt, const float* b_txt, const float* gq,
                              const float* gk, int B, int H, int N_img, int N_txt, int d, int C, jattn_bf16* q,
                              jattn_bf16* k, jattn_bf16* v, void* saved, void* stream) {
  return qkv_body(QkvCall{{x_img, x_txt}, {w_img, w_txt}, {b_img, b_txt}, gq, gk, B, H, N_img, N_txt, d, C, q, k, v,
                          saved, stream});
}

extern "C" int jattn_qkv_norm_fp8(const uint8_t* x_img, const float* sx_img, const uint8_t* w_img,
                                  const float* sw_img, const float* b_img, const uint8_t* x_txt,
                                  const float* sx_txt, const uint8_t* w_txt, const float* sw_txt,
                                  const float* b_txt, const float* gq, const float* gk, int B, int H, int N_img,
                                  int N_txt, int d, int C, jattn_bf16* q, jattn_bf16* k, jattn_bf16* v, void* saved,
                                  void* stream) {
  QkvCall c{{x_img, x_txt}, {w_img, w_txt}, {b_img, b_txt}, gq, gk, B, H, N_img, N_txt, d, C, q, k, v, saved, stream};
  c.e4m3 = true;
  c.sx[0] = sx_img;
  c.sx[1] = sx_txt;
  c.sw[0] = sw_img;
  c.sw[1] = sw_txt;
  return qkv_body(c);
}

extern "C" size_t jattn_qkv_norm_lora_bytes(int B, int H, int N_img, int N_txt, int d, int rank) {
  Shape s;
  if (check_shape(B, H, N_img, N_txt, d, &s) != JATTN_OK || check_lora(rank) != JATTN_OK) return 0;
  return lora_u_bytes(static_cast<int64_t>(B) * N_img, rank) + lora_u_bytes(static_cast<int64_t>(B) * N_txt, rank);
}

extern "C" int jattn_qkv_norm_lora(const jattn_bf16* x_img, const jattn_bf16* w_img, const float* b_img,
                                   const jattn_bf16* x_txt, const jattn_bf16* w_txt, const float* b_txt,
                                   const float* gq, const float* gk, const jattn_bf16* down_img,
                                   const jattn_bf16* up_img, const jattn_bf16* down_txt, const jattn_bf16* up_txt,
                                   const float* scale, const int* index, int n_adapters, int rank, int B, int H,
                                   int N_img, int N_txt, int d, int C, jattn_bf16* q, jattn_bf16* k, jattn_bf16* v,
                                   void* saved, void* work, void* stream) {
  QkvCall c{{x_img, x_txt}, {w_img, w_txt}, {b_img, b_txt}, gq, gk, B, H, N_img, N_txt, d, C, q, k, v, saved, stream};
  c.lora = true;
  c.down[0] = down_img;
  c.down[1] = down_txt;
  c.up[0] = up_img;
  c.up[1] = up_txt;
  c.scale = scale;
  c.index = index;
  c.n_adapters = n_adapters;
  c.rank = rank;
  c.work = work;
  return qkv_body(c);
}

extern "C" int jattn_fwd_saved(const jattn_bf16* v, int B, int H, int N_img, int N_txt, int d, jattn_bf16* out,
                               float* lse, void* saved, void* stream) {
  if (!v || !out || !lse || !saved) return JATTN_ERR_INVALID_ARG;
  Shape s;
  int rc = check_shape(B, H, N_img, N_txt, d, &s);
  if (rc != JATTN_OK) return rc;
  const void* ptrs[] = {v, out, lse, saved};
  for (const void* p : ptrs)
    if (!aligned16(p)) return JATTN_ERR_MISALIGNED;
  const size_t tb = s.elems * 2;
  const SavedLayout sl = saved_layout(s);
  const Range ins[] = {range_of(v, tb), range_of(saved, sl.total)};
  const Range outs[] = {range_of(out, tb), range_of(lse, s.rows * 4)};
  for (size_t a = 0; a < sizeof(outs) / sizeof(outs[0]); ++a) {
    for (const Range& i : ins)
      if (overlaps(outs[a], i)) return JATTN_ERR_ALIAS;
    for (size_t b = a + 1; b < sizeof(outs) / sizeof(outs[0]); ++b)
      if (overlaps(outs[a], outs[b])) return JATTN_ERR_ALIAS;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t* err = dev_err_ptr();
  if (!err) return fail(JATTN_ERR_CUDA, "device error word", cudaGetLastError());
  uint8_t* base = static_cast<uint8_t*>(saved);
  CUtensorMap mq, mk, mv;
  if (!encode_bhnd_map(&mq, base + sl.qhat, s.BH, s.N, s.d) || !encode_bhnd_map(&mk, base + sl.khat, s.BH, s.N, s.d) ||
      !encode_bhnd_map(&mv, v, s.BH, s.N, s.d))
    return fail(JATTN_ERR_CUDA, "cuTensorMapEncodeTiled");
  AttnShape as{s.BH, s.N, s.d, 1.0f / sqrtf(static_cast<float>(s.d)), s.seg};
  cudaError_t ce;
  {
    Timed t(JATTN_KERNEL_ATTN_FWD, st);
    ce = launch_attn_fwd(mq, mk, mv, as, out, lse, err, st, reinterpret_cast<float*>(base + sl.dq),
                         reinterpret_cast<uint32_t*>(base + sl.zero_count));
  }
  if (ce != cudaSuccess) return fail(JATTN_ERR_CUDA, "attn_fwd launch", ce);
  return JATTN_OK;
}

namespace {

int check_rows(int T, int C) {
  if (T <= 0 || C <= 0) return JATTN_ERR_INVALID_ARG;
  return C % 8 != 0 || C > JATTN_MAX_WIDTH ? JATTN_ERR_UNSUPPORTED : JATTN_OK;
}

// Any output over an input or another output; `same` (an output) may be
// exactly `as` (an input): those elements are read by the thread that
// overwrites them, before it does.
template <size_t I, size_t O>
bool any_alias(const Range (&ins)[I], const Range (&outs)[O], Range same, Range as) {
  auto equal = [](Range a, Range b) { return a.lo == b.lo && a.hi == b.hi; };
  for (size_t a = 0; a < O; ++a) {
    for (const Range& i : ins)
      if (overlaps(outs[a], i) && !(equal(outs[a], same) && equal(i, as) && equal(outs[a], i))) return true;
    for (size_t b = a + 1; b < O; ++b)
      if (overlaps(outs[a], outs[b])) return true;
  }
  return false;
}

// y (bf16) or y8 and s, exactly one of the two; g null: jattn_quant_rows.
int add_norm_body(const jattn_bf16* x, const jattn_bf16* res, const float* g, int T, int C, float eps, jattn_bf16* h,
                  jattn_bf16* y, uint8_t* y8, float* s, float* r, int kind, void* stream) {
  const int rc = check_rows(T, C);
  if (rc != JATTN_OK) return rc;
  const void* ptrs[] = {x, res, g, h, y, y8, s, r};
  for (const void* p : ptrs)
    if (!aligned16(p)) return JATTN_ERR_MISALIGNED;
  const size_t n = static_cast<size_t>(T) * C, rows = static_cast<size_t>(T) * 4;
  const Range ins[] = {range_of(x, n * 2), range_of(res, res ? n * 2 : 0), range_of(g, g ? C * sizeof(float) : 0)};
  const Range outs[] = {range_of(h, h ? n * 2 : 0), range_of(y, y ? n * 2 : 0), range_of(y8, y8 ? n : 0),
                        range_of(s, s ? rows : 0), range_of(r, r ? rows : 0)};
  if (any_alias(ins, outs, outs[0], ins[1])) return JATTN_ERR_ALIAS;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t ce;
  {
    Timed t(kind, st);
    ce = launch_add_norm(TokenNorm{x, res, g, T, C, eps, h, y, y8, s, r}, st);
  }
  if (ce != cudaSuccess) return fail(JATTN_ERR_CUDA, "token row kernel launch", ce);
  return JATTN_OK;
}

bool eps_ok(float eps) { return eps > 0.f && eps <= 3.402823466e38f; }

}  // namespace

extern "C" int jattn_add_norm(const jattn_bf16* x, const jattn_bf16* res, const float* g, int T, int C, float eps,
                              jattn_bf16* h, jattn_bf16* y, float* r, void* stream) {
  if (!x || !g || !y || (res == nullptr) != (h == nullptr) || !eps_ok(eps)) return JATTN_ERR_INVALID_ARG;
  return add_norm_body(x, res, g, T, C, eps, h, y, nullptr, nullptr, r, JATTN_KERNEL_ADD_NORM, stream);
}

extern "C" int jattn_add_norm_fp8(const jattn_bf16* x, const jattn_bf16* res, const float* g, int T, int C,
                                  float eps, jattn_bf16* h, uint8_t* y8, float* s, float* r, void* stream) {
  if (!x || !g || !y8 || !s || (res == nullptr) != (h == nullptr) || !eps_ok(eps)) return JATTN_ERR_INVALID_ARG;
  return add_norm_body(x, res, g, T, C, eps, h, nullptr, y8, s, r, JATTN_KERNEL_ADD_NORM, stream);
}

extern "C" int jattn_quant_rows(const jattn_bf16* x, int T, int C, uint8_t* x8, float* s, void* stream) {
  if (!x || !x8 || !s) return JATTN_ERR_INVALID_ARG;
  return add_norm_body(x, nullptr, nullptr, T, C, 0.f, nullptr, nullptr, x8, s, nullptr, JATTN_KERNEL_QUANT_ROWS,
                       stream);
}

extern "C" size_t jattn_add_norm_bwd_bytes(int T, int C) {
  if (check_rows(T, C) != JATTN_OK) return 0;
  return static_cast<size_t>(add_norm_bwd_parts(T, C)) * C * sizeof(float);
}

extern "C" int jattn_add_norm_bwd(const jattn_bf16* dy, const jattn_bf16* dh, const jattn_bf16* h, const float* r,
                                  const float* g, int T, int C, jattn_bf16* dx, float* dg, void* work,
                                  void* stream) {
  if (!dy || !h || !r || !g || !dx || !dg || !work) return JATTN_ERR_INVALID_ARG;
  const int rc = check_rows(T, C);
  if (rc != JATTN_OK) return rc;
  const void* ptrs[] = {dy, dh, h, r, g, dx, dg, work};
  for (const void* p : ptrs)
    if (!aligned16(p)) return JATTN_ERR_MISALIGNED;
  const size_t tb = static_cast<size_t>(T) * C * 2, gb = static_cast<size_t>(C) * 4;
  const Range ins[] = {range_of(dy, tb), range_of(dh, dh ? tb : 0), range_of(h, tb),
                       range_of(r, static_cast<size_t>(T) * 4), range_of(g, gb)};
  const Range outs[] = {range_of(dx, tb), range_of(dg, gb), range_of(work, jattn_add_norm_bwd_bytes(T, C))};
  if (any_alias(ins, outs, outs[0], ins[1])) return JATTN_ERR_ALIAS;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* part = static_cast<float*>(work);
  const int parts = add_norm_bwd_parts(T, C);
  cudaError_t ce;
  {
    Timed t(JATTN_KERNEL_ADD_NORM_BWD, st);
    ce = launch_add_norm_bwd(dy, dh, h, r, g, T, C, dx, part, parts, st);
  }
  if (ce != cudaSuccess) return fail(JATTN_ERR_CUDA, "add_norm_bwd launch", ce);
  {
    Timed t(JATTN_KERNEL_ADD_NORM_DG, st);
    ce = launch_dg_sum(part, parts, C, dg, st);
  }
  if (ce != cudaSuccess) return fail(JATTN_ERR_CUDA, "add_norm_dg launch", ce);
  return JATTN_OK;
}

namespace jattn {

// One thread waits on an mbarrier that nothing arrives at, through the same
// bounded wait the attention kernels use: it gives up after kWaitLimitNs and
// records DEV_ERR_WAIT_TIMEOUT, and the kernel returns.
__global__ void selftest_wait_kernel(uint32_t* dev_err) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x != 0) return;
  abort_flag = 0;
  mbar_init(&bar, 1);
  fence_mbar_init();
  mbar_wait(&bar, 0u, &abort_flag, dev_err);
}

}  // namespace jattn

extern "C" int jattn_selftest_wait_timeout(void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t* err = dev_err_ptr();
  if (!err) return fail(JATTN_ERR_CUDA, "device error word");
  jattn::selftest_wait_kernel<<<1, 32, 0, st>>>(err);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(JATTN_ERR_CUDA, "selftest_wait_kernel launch", e);
  return JATTN_OK;
}

extern "C" int jattn_last_device_error(void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(st) != cudaSuccess) return JATTN_ERR_CUDA;
  uint32_t* p = dev_err_ptr();
  if (!p) return JATTN_ERR_CUDA;
  uint32_t v = 0;
  if (cudaMemcpy(&v, p, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return JATTN_ERR_CUDA;
  if (v == 0) return JATTN_OK;
  const uint32_t zero = 0;
  if (cudaMemcpy(p, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess) return JATTN_ERR_CUDA;
  return (v & DEV_ERR_WAIT_TIMEOUT) ? JATTN_ERR_TIMEOUT : JATTN_ERR_CUDA;
}

extern "C" int jattn_profile_enable(int on) {
  Prof& p = prof();
  std::lock_guard<std::mutex> lock(p.mu);
  p.on = on != 0;
  return JATTN_OK;
}

extern "C" int jattn_profile_reset(void) {
  Prof& p = prof();
  std::lock_guard<std::mutex> lock(p.mu);
  int status = JATTN_OK;
  for (auto& r : p.pending) {
    if (cudaEventSynchronize(r.b) != cudaSuccess) status = JATTN_ERR_CUDA;
    p.pool.push_back(r.a);
    p.pool.push_back(r.b);
  }
  p.pending.clear();
  for (int i = 0; i < JATTN_TOKEN_KERNEL_END; ++i) {
    p.launches[i] = 0;
    p.ms[i] = 0;
  }
  return status;
}

extern "C" int jattn_profile_read(int kind, int* launches, double* total_ms) {
  const bool known = (kind >= 0 && kind < JATTN_KERNEL_COUNT) ||
                     (kind >= JATTN_TOKEN_KERNEL_FIRST && kind < JATTN_TOKEN_KERNEL_END);
  if (!known || !launches || !total_ms) return JATTN_ERR_INVALID_ARG;
  Prof& p = prof();
  std::lock_guard<std::mutex> lock(p.mu);
  int status = JATTN_OK;
  for (auto& r : p.pending) {
    float ms = 0.f;
    if (cudaEventSynchronize(r.b) != cudaSuccess || cudaEventElapsedTime(&ms, r.a, r.b) != cudaSuccess) {
      status = JATTN_ERR_CUDA;
    } else {
      p.launches[r.kind] += 1;
      p.ms[r.kind] += ms;
    }
    p.pool.push_back(r.a);
    p.pool.push_back(r.b);
  }
  p.pending.clear();
  *launches = static_cast<int>(p.launches[kind]);
  *total_ms = p.ms[kind];
  return status;
}

extern "C" int jattn_set_deterministic(int on) {
  g_deterministic.store(on != 0 ? 1 : 0, std::memory_order_relaxed);
  return JATTN_OK;
}

extern "C" int jattn_set_sm_limit(int max_sms) {
  if (max_sms < 0) return JATTN_ERR_INVALID_ARG;
  set_sm_limit(max_sms);
  return JATTN_OK;
}

extern "C" const char* jattn_kernel_name(int kind) {
  switch (kind) {
    case JATTN_KERNEL_QK_NORM_FWD: return "qk_norm_fwd";
    case JATTN_KERNEL_ATTN_FWD: return "attn_fwd";
    case JATTN_KERNEL_BWD_PREP: return "bwd_prep";
    case JATTN_KERNEL_ATTN_BWD: return "attn_bwd";
    case JATTN_KERNEL_Q_NORM_BWD: return "q_norm_bwd";
    case JATTN_KERNEL_QKV_NORM: return "qkv_norm";
    case JATTN_KERNEL_ADD_NORM: return "add_norm";
    case JATTN_KERNEL_ADD_NORM_BWD: return "add_norm_bwd";
    case JATTN_KERNEL_ADD_NORM_DG: return "add_norm_dg";
    case JATTN_KERNEL_QUANT_ROWS: return "quant_rows";
    case JATTN_KERNEL_LORA_DOWN: return "lora_down";
    default: return "unknown";
  }
}

extern "C" const char* jattn_status_string(int status) {
  switch (status) {
    case JATTN_OK: return "ok";
    case JATTN_ERR_INVALID_ARG: return "invalid argument (null pointer, non-positive or overflowing size)";
    case JATTN_ERR_UNSUPPORTED:
      return "unsupported size (d must be 64 or 128; C a multiple of 8, or of 16 for 8-bit tokens, and for token "
             "rows at most 16384; a rank a multiple of 8, at most 128)";
    case JATTN_ERR_MISALIGNED: return "pointer not 16-byte aligned";
    case JATTN_ERR_ALIAS: return "an output buffer overlaps another buffer";
    case JATTN_ERR_CUDA: return "CUDA launch or allocation failed";
    case JATTN_ERR_TIMEOUT: return "device-side bounded wait timed out";
    case JATTN_ERR_SCRATCH_LIMIT: return "problem needs more scratch than the fixed no-alloc array holds";
    default: return "unknown status";
  }
}

extern "C" int jattn_version(void) { return kVersion; }

extern "C" const char* jattn_last_error_message(void) { return g_last_msg; }
