// qkv_lora.cu — the QKV projection with low-rank adapters of the batch items'
// own (qkv_proj.cuh), and the adapters' first product.
#include "qkv_proj.cuh"

namespace jattn {
namespace {

// U = scale X A^T.
// One CTA per batch item, stream and block of 128 of its token rows: an item
// has one adapter, whose down weights [3 rank, C] are the product's other
// operand, N = 3 * 16 rank_units columns (a rank that is not a multiple of 16
// reads the TMA's zero fill).  Items without an adapter write nothing (the
// projection reads nothing of theirs).  U is kept as three bf16 terms, each what
// the ones before leave rounded: together they are the fp32 value, so that Y has
// one rounding.  Of 10 000 values of q 4.5 are not the bf16 value nearest to the
// exact one (512 px, rank 16), 4.1 without adapters; with two terms, which lose up
// to 2^-17 of U, 8.4 were (and a call took 65.8 us instead of 66.4, of rank 128 110
// instead of 119).  Warps 0-3 read the accumulator out (a row a thread), warp 4
// loads, warp 5 issues.
//
// What bounds it: its own start and end.  At 512 px (16 items, rank 16) it reads
// 27 MB in 13 us under ncu, with 4 stages of the ring as with 12; the projection
// starts behind its first wait, so that the call takes 66 us where the
// projection alone takes 52 and, with no item having an adapter, 55.
constexpr int kDownThreads = 192;
constexpr int kDownK = 64;
constexpr int kDownMaxStages = 6;
constexpr int kDownSmem = 200 * 1024;

struct DownStream {
  int N_s, blocks, cta0;  // rows per item, its 128-row blocks, the stream's first CTA
  uint16_t* u;            // [B N_s, 3 rank_units, 3, 16]: the first terms of 16 values, the second, the third
};
struct DownParams {
  DownStream s[2];
  int C, rank_units, n_adapters, stages, tmem_cols;
  bool half_unit;  // the rank is an odd multiple of 8: the last unit's second half stands for nothing
  const int* index;
  const float* scale;
};
struct DownMaps {
  CUtensorMap x[2], down[2];  // [B, N_s, C] with 128-row boxes; [3 n, rank, C] with 16 rank_units rows
};
struct DownBars {
  uint64_t full[kDownMaxStages], empty[kDownMaxStages], done;
  uint32_t tmem_base;
  int abort;
};

__global__ void __launch_bounds__(kDownThreads, 1)
    lora_down_kernel(const __grid_constant__ DownMaps maps, const __grid_constant__ DownParams p,
                     uint32_t* dev_err) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) DownBars bars;
  uint8_t* sm = align1024(smem_raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* ab = &bars.abort;
  // The projection may start once every CTA is past this wait: what came before
  // this kernel is then complete, and only U is still to come (it waits for it).
  griddep_wait();
  griddep_launch_dependents();
  const int si = static_cast<int>(blockIdx.x) >= p.s[1].cta0 ? 1 : 0;
  const int N_s = si ? p.s[1].N_s : p.s[0].N_s, blocks = si ? p.s[1].blocks : p.s[0].blocks;
  const int local = blockIdx.x - (si ? p.s[1].cta0 : p.s[0].cta0);
  const int item = local / blocks, row0 = (local - item * blocks) * kBM;
  const int adapter = __ldg(p.index + item);
  if (adapter < 0 || adapter >= p.n_adapters) return;  // the whole CTA
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    mbar_init(&bars.done, 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc<1>(&bars.tmem_base, p.tmem_cols);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  const int ksteps = (p.C + kDownK - 1) / kDownK;
  const int r16 = 16 * p.rank_units;
  const int stage_bytes = kATile + 3 * r16 * 128;
  if (warp == 4) {
    if (lane == 0) {
      const CUtensorMap* mx = si ? &maps.x[1] : &maps.x[0];
      const CUtensorMap* md = si ? &maps.down[1] : &maps.down[0];
      int kb = 0;
      for (; kb < ksteps; ++kb) {
        const int s = kb % p.stages;
        if (kb >= p.stages && !mbar_wait(&bars.empty[s], ((kb / p.stages) - 1) & 1, ab, dev_err)) break;
        uint8_t* st = sm + s * stage_bytes;
        mbar_arrive_expect_tx(&bars.full[s], stage_bytes);
        tma_load_3d(st, mx, &bars.full[s], kb * kDownK, row0, item);
        for (int part = 0; part < 3; ++part)
          tma_load_3d(st + kATile + part * r16 * 128, md, &bars.full[s], kb * kDownK, 0, 3 * adapter + part);
      }
      if (*ab)  // aborted: the copies in flight land before the CTA exits
        drain_ring(kb, p.stages, true, [&](int s, uint32_t parity) { mbar_wait_drain(&bars.full[s], parity); });
    }
  } else if (warp == 5) {
    if (lane == 0) {
      const bool one = 3 * r16 <= 256;
      const uint32_t idesc = idesc_bf16_f32(kBM, one ? 3 * r16 : r16, false, false);
      for (int kb = 0; kb < ksteps; ++kb) {
        const int s = kb % p.stages;
        if (!mbar_wait(&bars.full[s], (kb / p.stages) & 1, ab, dev_err)) break;
        tc_fence_after();
        const uint32_t st = smem_u32(sm + s * stage_bytes);
        const uint64_t a = sdesc_sw128(st, 16, 1024), b = sdesc_sw128(st + kATile, 16, 1024);
        for (int kk = 0; kk < kDownK / 16; ++kk) {
          const uint32_t add = (kb > 0 || kk > 0) ? 1u : 0u;
          for (int part = 0; part < (one ? 1 : 3); ++part)
            umma_bf16_ss<1>(tmem + part * r16, desc_add(a, kk * 32), desc_add(b, kk * 32 + part * r16 * 128), idesc,
                         add);
        }
        umma_commit<1>(&bars.empty[s]);
      }
      // Every MMA this thread issued has completed once this barrier flips.
      umma_commit<1>(&bars.done);
      mbar_wait_drain(&bars.done, 0);
    }
  } else {
    bool ok = mbar_wait(&bars.done, 0, ab, dev_err);
    ok = __all_sync(0xffffffffu, ok) && !*ab;
    __syncwarp();
    if (__all_sync(0xffffffffu, ok)) {
      tc_fence_after();
      const float scale = __ldg(p.scale + adapter);
      const int n = row0 + warp * 32 + lane;
      uint16_t* u = (si ? p.s[1].u : p.s[0].u) + (static_cast<size_t>(item) * N_s + n) * (9 * r16);
      for (int c = 0; c < 3 * p.rank_units; ++c) {
        uint32_t v[16];
        tmem_ld16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c * 16, v);
        tmem_wait_ld();
        // Each remainder is exact in fp32.  The first two terms end at the largest bf16 value, so that a value
        // above it keeps its rest and an infinity is the last term (not inf - inf).
        uint32_t w[3][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float a = __uint_as_float(v[2 * i]) * scale, b = __uint_as_float(v[2 * i + 1]) * scale;
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            w[k][i] = k < 2 ? pack_bf16x2_sat(a, b) : pack_bf16x2(a, b);
            a -= bf_lo(w[k][i]);
            b -= bf_hi(w[k][i]);
          }
        }
        if (p.half_unit && c % p.rank_units == p.rank_units - 1) {  // past the rank: 0, for infinite tokens too
#pragma unroll
          for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int i = 4; i < 8; ++i) w[k][i] = 0u;
        }
        if (n < N_s) {
          uint4* o = reinterpret_cast<uint4*>(u + c * 48);
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            o[2 * k] = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
            o[2 * k + 1] = make_uint4(w[k][4], w[k][5], w[k][6], w[k][7]);
          }
        }
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, p.tmem_cols);
  }
}

}  // namespace

cudaError_t launch_lora_down(const CUtensorMap (&x)[2], const CUtensorMap (&down)[2], const LoraLaunch& l,
                             const QkvLaunch& a, int B, uint32_t* dev_err, cudaStream_t st) {
  DownMaps maps;
  DownParams p;
  const int r16 = (l.rank + 15) / 16 * 16;
  int ctas = 0;
  for (int i = 0; i < 2; ++i) {
    maps.x[i] = x[i];
    maps.down[i] = down[i];
    p.s[i].N_s = a.N_s[i];
    p.s[i].blocks = l.on[i] ? (a.N_s[i] + kBM - 1) / kBM : 0;
    p.s[i].cta0 = ctas;
    p.s[i].u = l.u[i];
    ctas += B * p.s[i].blocks;
  }
  if (ctas == 0) return cudaSuccess;
  p.C = a.C;
  p.rank_units = r16 / 16;
  p.half_unit = l.rank % 16 != 0;
  p.n_adapters = l.n_adapters;
  const int stage_bytes = kATile + 3 * r16 * 128;
  p.stages = kDownSmem / stage_bytes < kDownMaxStages ? kDownSmem / stage_bytes : kDownMaxStages;
  p.tmem_cols = 32;
  while (p.tmem_cols < 3 * r16) p.tmem_cols *= 2;
  p.index = l.index;
  p.scale = l.scale;
  const int smem = p.stages * stage_bytes + 1024;
  // The limit for every rank: a call of another thread, or a captured one, may be of a higher rank.
  cudaError_t e = cudaFuncSetAttribute(lora_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kDownSmem + 1024);
  if (e != cudaSuccess) return e;
  return launch_pdl(lora_down_kernel, dim3(ctas), dim3(kDownThreads), smem, st, maps, p, dev_err);
}

cudaError_t launch_qkv_norm_lora(const CUtensorMap (&maps)[4], const QkvLaunch& a,
                                 uint32_t* dev_err, cudaStream_t st, const LoraLaunch* lora,
                                 const CUtensorMap* lora_maps) {
  return launch_qkv_form<kLora>(maps, a, dev_err, st, lora, lora_maps);
}

}  // namespace jattn
