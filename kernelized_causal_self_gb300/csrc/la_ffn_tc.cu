// The gated projections in bf16 on the tensor cores: a = x wg^T, u = x wu^T, h = act(a) u, and
// the backward pass da = dh u act'(a), du = dh act(a), dx = da wg + du wu, dwg = da^T x,
// dwu = du^T x (da and du in bf16, in the workspace). da and du have to be bf16 for the tensor cores to
// multiply them: a second term of each would double the sums' multiplications, two thirds of the whole.
// It costs half a step, 2^-8, of every factor: dx, dwg, dwu of random data are 2.35e-3 off in the
// 2-norm where results of float32 factors, rounded themselves, are 1.66e-3.
//
// One persistent kernel for all five products (in two launches, dx and the weights' in one). A
// pair of CTAs (cta_group::2) makes a tile of 256 x 256: each CTA copies its 128 rows of A and its
// half of B's 256 rows by TMA, 64 terms of the sum a stage, the even one issues the MMAs, and each finds its 128 x 256 of D in its
// own tensor memory, where two accumulators take turns, so that eight warps write one tile's
// results while the next is summed.
//   kForward, kGrads  A = x, B = 128 rows of wg (even CTA) and the same rows of wu (odd CTA): a
//                     row's a and u come to lie in one thread, 128 columns apart, and nothing
//                     but h (or da, du) leaves the SM. kGrads has dh's tile copied in as well.
//   kSums, dx         A = [da | du], B = [wg; wu] read along c: one sum over 2 F terms.
//   kSums, dwg, dwu   A = da or du and B = x, both read along their rows (tokens are the sum).
// Results go through a swizzled staging tile of 32 rows a warp and leave by TMA, which clips
// what is past the matrix; copies past its edge read zeros, so ragged sizes need no masks.
// Sums with few tiles, or of many terms, are cut along k (float32 parts, added in order by a second kernel).
//
// Bound by the tensor cores, and by shared memory's bandwidth where a value's results are many
// (operands alone take most of it). T 65536, C 512, F 1408: h in 115 us (1640 TFLOP/s; 131 under the
// power limit), da and du in 148, dx, dwg and dwu in 232 (1630 TFLOP/s); T 4096, C 2048, F 5632: h in 105
// to 113, 128 with a checkpoint.
#include <cuda_bf16.h>

#include "la_ffn_tc.cuh"

namespace la {
namespace {

using namespace ffn;

// one more warp that copies, one that multiplies, kGrads: one that copies dh
constexpr int threads_of(int kind) { return 32 * (kWarps + (kind == kGrads ? 3 : 2)); }
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int stages_of(int kind) { return kind == kGrads ? 4 : 6; }
constexpr int smem_of(int kind) {
  return 1024 + stages_of(kind) * kStageBytes + kWarps * kStore + (kind == kGrads ? 4 * kTileBytes : 0) + 256;
}

struct Args : Grids {
  CUtensorMap a, b0, b1;         // operands: x or da, du; wg; wu
  CUtensorMap aw, bw;            // of dwg and dwu: da, du and x, both read along their rows
  CUtensorMap out0, out1, out2;  // h; da, du; dx, dwg, dwu. Of cut sums their parts in float32: out0
                                 // [splits][T][C], out1 [2][splits][F][C]
  CUtensorMap dh;                // kGrads
  WorkspaceHeader* hdr;
  signed char* codes;            // kForward: a checkpoint of a, u
  unsigned char* exps;
  int clear;                     // the call's first kernel clears the status header
};

template <int KIND, int ACT>
__global__ void __launch_bounds__(threads_of(KIND), 1) ffn_tc_kernel(const __grid_constant__ Args a) {
  constexpr int S = stages_of(KIND);
  constexpr bool DUAL = KIND == kForward || KIND == kGrads;
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
  uint8_t* stages = sm;                                  // [stage][A | B]
  uint8_t* dht = stages + S * kStageBytes;               // kGrads: dh's tiles, two in turn, each two
                                                         // blocks of 64 columns
  uint8_t* staging = dht + (KIND == kGrads ? 4 * kTileBytes : 0);
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kWarps * kStore);  // S (the even CTA's count)
  uint64_t* empty = full + S;                            // S: the MMAs are done with the stage
  uint64_t* acc_full = empty + S;                        // 2: an accumulator holds its tile
  uint64_t* acc_empty = acc_full + 2;                    // 2 (the even CTA's): both CTAs have read it
  uint64_t* dh_full = acc_empty + 2;                     // 2
  uint64_t* dh_empty = dh_full + 2;                      // 2: du, which took dh's place, has left
  uint64_t* drain = dh_empty + 2;
  volatile int* abort = reinterpret_cast<volatile int*>(drain + 1);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 1) + 1;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const int cluster = blockIdx.x / 2, clusters = gridDim.x / 2;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kWarps);
      mbar_init(&dh_full[b], 1);
      mbar_init(&dh_empty[b], kWarps);
    }
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc_pair(tslot, 512);
    tmem_relinquish_pair();
  }
  if (warp == kWarps && lane == 0) {
    prefetch_tensormap(&a.a);
    prefetch_tensormap(&a.b0);
    prefetch_tensormap(&a.out0);
    prefetch_tensormap(&a.b1);
    if (KIND == kGrads) prefetch_tensormap(&a.dh);
    if (KIND != kForward) prefetch_tensormap(&a.out1);
    if (KIND == kSums) {
      prefetch_tensormap(&a.aw);
      prefetch_tensormap(&a.bw);
    }
  }
  fence_before_sync();
  __syncthreads();
  cluster_sync();
  fence_after_sync();
  const uint32_t tbase = *tslot;
  pdl_wait();
  WorkspaceHeader* hdr = a.hdr;
  // (a wait that runs out is recorded two seconds after its kernel began, long after this)
  if (a.clear && blockIdx.x == 0 && threadIdx.x == 0) hdr->status = hdr->wait_site = 0;

  if (warp == kWarps) {
    // ------------------------------------------------------------------ copies
    if (lane == 0) {
      const uint32_t bars = cluster_map(smem_u32(full), 0);
      uint32_t s = 0, phase = 1;  // (a stage not used yet counts as emptied once)
      bool ok = true;
      for (int t, i = 0; ok && (t = dealt<KIND>(a, cluster, clusters, i)) >= 0; ++i) {
        const Tile w = tile_of<KIND>(a, t);
        const Grid& g = a.g[w.dw];
        const int row = w.m * 256 + (int)rank * 128, end = first_step(g, w.split + 1);
        if (DUAL && t + clusters < g.tiles) {
          // x of the next tile into L2, a tile's time ahead: the tiles of the same rows share its steps
          const Tile v = tile_of<KIND>(a, t + clusters);
          for (int k = v.n; k < g.steps; k += g.n_tiles) tma_prefetch_3d(&a.a, k * 64, v.m * 256 + (int)rank * 128, 0);
        }
        for (int k = first_step(g, w.split); k < end; ++k) {
          if (!mbar_wait_abort(&empty[s], phase, abort, hdr, kSiteEmpty)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kStageBytes);
          const uint32_t bar = bars + 8 * s;
          uint8_t *ta = stages + s * kStageBytes, *tb = ta + kTileBytes;
          if constexpr (DUAL) {
            tma_load_3d_pair(ta, &a.a, bar, k * 64, row, 0);
            tma_load_3d_pair(tb, rank ? &a.b1 : &a.b0, bar, k * 64, w.n * 128, 0);
          } else if (!w.dw) {
            const int part = k >= g.per, kk = (part ? k - g.per : k) * 64;
            const int col = w.n * 256 + (int)rank * 128;
            tma_load_3d_pair(ta, &a.a, bar, kk, row, part);
            tma_load_3d_pair(tb, part ? &a.b1 : &a.b0, bar, col, kk, 0);
            tma_load_3d_pair(tb + kTileBytes / 2, part ? &a.b1 : &a.b0, bar, col + 64, kk, 0);
          } else {
            const int col = w.n * 256 + (int)rank * 128;
            tma_load_3d_pair(ta, &a.aw, bar, row, k * 64, w.part);
            tma_load_3d_pair(ta + kTileBytes / 2, &a.aw, bar, row + 64, k * 64, w.part);
            tma_load_3d_pair(tb, &a.bw, bar, col, k * 64, 0);
            tma_load_3d_pair(tb + kTileBytes / 2, &a.bw, bar, col + 64, k * 64, 0);
          }
          if (++s == S) s = 0, phase ^= 1;
        }
      }
      // A CTA lets go of its shared memory once its last stages are multiplied and every commit to it has
      // come in; if a wait ran out, once the pair's copies have landed. (Stages before s were used
      // in this turn, the others in the one before.)
      for (uint32_t k = 0; k < S; ++k) {
        const uint32_t turn = k < s ? phase ^ 1 : phase;
        if (ok ? !mbar_wait(&empty[k], turn) : rank == 0 && !mbar_wait(&full[k], turn)) record_timeout(hdr, kSiteDrain);
      }
    }
    __syncwarp();
  } else if (KIND == kGrads && warp == kWarps + 2) {
    // ------------------------------------------------------------------ dh's tiles
    // (a thread of its own: its wait for the results to be out holds up no operand)
    if (lane == 0) {
      int nt = 0;
      bool ok = true;
      for (int t; (t = dealt<KIND>(a, cluster, clusters, nt)) >= 0;) {
        const Tile w = tile_of<KIND>(a, t);
        const int row = w.m * 256 + (int)rank * 128;
        const int b = nt & 1;
        if (nt >= 2) ok = mbar_wait_abort(&dh_empty[b], (uint32_t)((nt / 2 - 1) & 1), abort, hdr, kSiteDhEmpty);
        if (!ok) break;
        mbar_arrive_expect_tx(&dh_full[b], 2 * kTileBytes);
        tma_load_3d(dht + 2 * b * kTileBytes, &a.dh, &dh_full[b], w.n * 128, row, 0);
        tma_load_3d(dht + (2 * b + 1) * kTileBytes, &a.dh, &dh_full[b], w.n * 128 + 64, row, 0);
        ++nt;
      }
      for (int t = nt > 2 ? nt - 2 : 0; t < nt; ++t)
        if (!mbar_wait(&dh_full[t & 1], (uint32_t)(t / 2 & 1))) record_timeout(hdr, kSiteDrain);
    }
    __syncwarp();
  } else if (warp == kWarps + 1) {
    // ------------------------------------------------------------------ products
    if (lane == 0 && rank == 0) {
      // along k: 32 bytes of a row a step of 16; along m or n: 16 rows, blocks of 64 columns 8 KB apart
      const uint32_t at = smem_u32(stages);
      const uint64_t da_k = sdesc(at, 16, 1024), da_m = sdesc(at, kTileBytes / 2, 1024);
      const uint64_t db0 = DUAL ? sdesc(at + kTileBytes, 16, 1024) : sdesc(at + kTileBytes, kTileBytes / 2, 1024);
      constexpr uint32_t ALONG_K = 32 / 16, ALONG_MN = 2048 / 16, STEP_B = DUAL ? ALONG_K : ALONG_MN;
      uint32_t s = 0, phase = 0;
      int nt = 0;
      bool ok = true;
      for (int t; ok && (t = dealt<KIND>(a, cluster, clusters, nt)) >= 0; ++nt) {
        int n = a.g[0].steps, dw = 0;
        if (!DUAL) {
          const Tile w = tile_of<KIND>(a, t);
          dw = w.dw;
          n = first_step(a.g[dw], w.split + 1) - first_step(a.g[dw], w.split);
        }
        const uint64_t da0 = !DUAL && dw ? da_m : da_k;
        const uint32_t step_a = !DUAL && dw ? ALONG_MN : ALONG_K;
        const uint32_t id = !DUAL && dw ? idesc_bf16(256, 256, true, true) : idesc_bf16(256, 256, false, !DUAL);
        const int b = nt & 1;
        if (nt >= 2) ok = mbar_wait_abort(&acc_empty[b], (uint32_t)((nt / 2 - 1) & 1), abort, hdr, kSiteAccEmpty);
        if (!ok) break;
        fence_after_sync();
        const uint32_t d = tbase + 256 * b;
        for (int k = 0; k < n; ++k) {
          if (!mbar_wait_abort(&full[s], phase, abort, hdr, kSiteFull)) {
            ok = false;
            break;
          }
          fence_after_sync();
          // (addresses are the descriptors' low bits, in units of 16 bytes)
          const uint64_t da = da0 + s * (kStageBytes / 16), db = db0 + s * (kStageBytes / 16);
#pragma unroll
          for (int q = 0; q < 4; ++q) mma_ss_pair(d, da + q * step_a, db + q * STEP_B, id, (k | q) != 0);
          mma_commit_pair(&empty[s]);
          if (++s == S) s = 0, phase ^= 1;
        }
        if (ok) mma_commit_pair(&acc_full[b]);
      }
      mma_commit_pair_own(drain);
      if (!mbar_wait(drain, 0)) record_timeout(hdr, kSiteDrain);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ results
    uint8_t* mine = staging + warp * kStore;
    const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
    const uint32_t freed = cluster_map(smem_u32(acc_empty), 0);
    constexpr int GROUPS = DUAL ? 1 : 2;    // of 64 columns
    int nt = 0;
    for (int t; (t = dealt<KIND>(a, cluster, clusters, nt)) >= 0; ++nt) {
      const Tile w = tile_of<KIND>(a, t);
      const Grid& grid = a.g[w.dw];
      const int b = nt & 1, row0 = w.m * 256 + (int)rank * 128 + warp % 4 * 32, row = row0 + lane;
      if (!mbar_wait_warp(&acc_full[b], (uint32_t)((nt / 2) & 1), abort, hdr, kSiteAccFull)) break;
      if (KIND == kGrads && !mbar_wait_warp(&dh_full[b], (uint32_t)(nt / 2 & 1), abort, hdr, kSiteDhFull)) break;
      fence_after_sync();
      const uint32_t d = tbase + 256 * b + lanes;
#pragma unroll 1
      for (int g = warp / 4 * GROUPS; g < (warp / 4 + 1) * GROUPS; ++g) {
        const int col = w.n * (DUAL ? 128 : 256) + g * 64;
        const bool cut = !DUAL && grid.splits > 1;
        uint8_t* st = mine;
        // kGrads: the warp's 32 rows of dh's block, where du takes dh's place, value by value
        uint8_t* dut = dht + (2 * b + g) * kTileBytes + warp % 4 * kStore;
        auto leave = [&](const CUtensorMap* to, int from, int mat) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (row0 < grid.rows && from < grid.cols) {
              tma_store_3d(to, st, from, row0, mat);
              if (KIND == kGrads) tma_store_3d(&a.out1, dut, from, row0, mat);
            }
            bulk_commit();
          }
        };
        auto left = [&]() {  // the last copy out of the staging tile has read it
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
        };
        if (!cut) left();
        if (KIND == kGrads && nt > 0 && lane == 0) mbar_arrive(&dh_empty[b ^ 1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // 32 columns
          uint32_t p[32], q[32];
          if constexpr (DUAL) {
            tmem_ld32x2(d + g * 64 + c * 32, p, d + 128 + g * 64 + c * 32, q);
            const float *fa = reinterpret_cast<const float*>(p), *fu = reinterpret_cast<const float*>(q);
            if constexpr (KIND == kForward) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int j = e * 8 + i * 2;
                  const float2 h = mul2(act2<ACT>(make_float2(fa[j], fa[j + 1])), make_float2(fu[j], fu[j + 1]));
                  o[i] = pack_bf16(h.x, h.y);
                }
                *reinterpret_cast<uint4*>(st + sw128(lane, c * 64 + e * 16)) = make_uint4(o[0], o[1], o[2], o[3]);
              }
              if (a.codes != nullptr) {  // a thread has a block of 32 of a and of u
                const int f = col + c * 32, nb = q8::blocks_of(grid.cols);
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                  const float* x = v ? fu : fa;
                  float top = fabsf(x[0]);
#pragma unroll
                  for (int j = 1; j < 31; j += 2) top = q8::top3(top, x[j], x[j + 1]);
                  const uint32_t e = q8::step_of(__float_as_uint(q8::top3(top, x[31], x[31])));
                  const float inv = q8::inverse_step(e);
                  if (row < grid.rows && f < grid.cols) {
                    const size_t r = 2 * (size_t)row + v;
                    signed char* to = a.codes + r * grid.cols + f;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                      if (f + j * 8 < grid.cols)
                        *reinterpret_cast<uint2*>(to + j * 8) =
                            make_uint2(q8::codes4(x + j * 8, inv, e), q8::codes4(x + j * 8 + 4, inv, e));
                    a.exps[r * nb + f / q8::kBlock] = (unsigned char)e;
                  }
                }
              }
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t at = sw128(lane, c * 64 + e * 16);
                const uint4 v = *reinterpret_cast<const uint4*>(dut + at);
                const uint32_t dh[4] = {v.x, v.y, v.z, v.w};
                uint32_t oa[4], ou[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int j = e * 8 + i * 2;
                  const float2 dv = make_float2(bf16_lo_f(dh[i]), bf16_hi_f(dh[i]));
                  float2 f, df;
                  act_grad2<ACT>(make_float2(fa[j], fa[j + 1]), f, df);
                  const float2 da = mul2(mul2(dv, make_float2(fu[j], fu[j + 1])), df), du = mul2(dv, f);
                  oa[i] = pack_bf16(da.x, da.y);
                  ou[i] = pack_bf16(du.x, du.y);
                }
                *reinterpret_cast<uint4*>(st + at) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
                *reinterpret_cast<uint4*>(dut + at) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
              }
            }
          } else {
            tmem_ld32(d + g * 64 + c * 32, p);
            if (cut) {  // 32 float32 are a staging row
              left();
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<uint4*>(st + sw128(lane, e * 16)) = make_uint4(p[4 * e], p[4 * e + 1], p[4 * e + 2], p[4 * e + 3]);
              leave(w.dw ? &a.out1 : &a.out0, col + c * 32, w.part * grid.splits + w.split);
            } else {
              const float* f = reinterpret_cast<const float*>(p);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *reinterpret_cast<uint4*>(st + sw128(lane, c * 64 + e * 16)) =
                    make_uint4(pack_bf16(f[e * 8], f[e * 8 + 1]), pack_bf16(f[e * 8 + 2], f[e * 8 + 3]),
                               pack_bf16(f[e * 8 + 4], f[e * 8 + 5]), pack_bf16(f[e * 8 + 6], f[e * 8 + 7]));
            }
          }
        }
        if (g % GROUPS == GROUPS - 1) {  // the accumulator may be written again
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(freed + 8 * b);
        }
        if (!cut) leave(!w.dw ? &a.out0 : w.part ? &a.out2 : &a.out1, col, 0);
      }
    }
    if (lane == 0) bulk_wait_all<0>();
    __syncwarp();
  }
  fence_before_sync();
  __syncthreads();
  cluster_sync();
  fence_after_sync();
  if (warp == 0) tmem_dealloc_pair(tbase, 512);
}

template <int KIND, int ACT>
cudaError_t launch(const Args& a, cudaStream_t st) {
  cudaError_t e = configure_once<ffn_tc_kernel<KIND, ACT>>(smem_of(KIND));
  if (e != cudaSuccess) return e;
  const int tiles = a.g[0].tiles + a.g[1].tiles;
  const int pairs = tiles < sm_count() / 2 ? tiles : sm_count() / 2;
  e = launch_cluster_pdl(ffn_tc_kernel<KIND, ACT>, dim3(2 * pairs), dim3(threads_of(KIND)), smem_of(KIND), st, 2, a);
  count_launches(1);
  return e;
}

template <int KIND>
cudaError_t launch_act(const Args& a, int act, cudaStream_t st) {
  return act == kSilu   ? launch<KIND, kSilu>(a, st)
         : act == kGelu ? launch<KIND, kGelu>(a, st)
                        : launch<KIND, kGeluTanh>(a, st);
}

// At most 32768 terms a part. The tensor cores' adder cuts off towards zero: a sum of n terms of one sign
// comes out n 4.6e-9 to n 6.2e-9 of itself too small (measured, 7.6e-5 of 16384, 1.6e-3 of 262144
// tokens, where half a step of bf16 is 3.9e-3), while parts are added in float32, rounded.
constexpr Costs kCosts{700, 4300, 512};

// a = x wg^T, u = x wu^T
bool products(Args& a, const FfnGate& f) {
  static_cast<Grids&>(a) = products_grid(f.T, f.C, f.F);
  a.clear = 1;
  return rows_map(&a.a, f.x, f.C, f.T, f.x_stride, 128) && rows_map(&a.b0, f.wg, f.C, f.F, f.C, 128) &&
         rows_map(&a.b1, f.wu, f.C, f.F, f.C, 128);
}

size_t dact_bytes(int T, int F) { return align_up(2 * sizeof(__nv_bfloat16) * (size_t)T * F, 256); }

}  // namespace

size_t ffn_tc_backward_workspace(int T, int C, int F) {
  const Grids& g = sums_grids(T, C, F, kCosts);
  return kHeaderBytes + dact_bytes(T, F) + sizeof(float) * (dx_parts(g) + dw_parts(g));
}

cudaError_t ffn_tc_forward(const FfnGate& f, void* ws, cudaStream_t st) {
  Args a{};
  a.hdr = static_cast<WorkspaceHeader*>(ws);
  a.codes = f.codes;
  a.exps = f.exps;
  if (!products(a, f) || !rows_map(&a.out0, f.h, f.F, f.T, f.h_stride, 32)) return cudaErrorInvalidValue;
  return launch_act<kForward>(a, f.act, st);
}

cudaError_t ffn_tc_backward(const FfnGate& f, void* ws, cudaStream_t st) {
  char* at = static_cast<char*>(ws) + kHeaderBytes;
  __nv_bfloat16 *da = reinterpret_cast<__nv_bfloat16*>(at), *du = da + (size_t)f.T * f.F;
  float* parts = reinterpret_cast<float*>(at + dact_bytes(f.T, f.F));
  Args a{};
  a.hdr = static_cast<WorkspaceHeader*>(ws);
  cudaError_t e;
  if (f.codes != nullptr || ffn_few(f.T, f.F, f.dtype)) {
    e = f.codes != nullptr ? ffn_kept_grads(f, da, st) : ffn_few_grads(f, da, st);
    a.clear = 1;
  } else {
    if (!products(a, f) || !rows_map(&a.dh, f.dh, f.F, f.T, f.dh_stride, 128) ||
        !rows_map(&a.out0, da, f.F, f.T, f.F, 32) || !rows_map(&a.out1, du, f.F, f.T, f.F, 32))
      return cudaErrorInvalidValue;
    e = launch_act<kGrads>(a, f.act, st);
    a.clear = 0;
  }
  if (e != cudaSuccess) return e;

  const Grids& g = sums_grids(f.T, f.C, f.F, kCosts);
  static_cast<Grids&>(a) = g;
  const int sx = g.g[0].splits, sw = g.g[1].splits;
  if (!rows_map(&a.a, da, f.F, f.T, f.F, 128, 2) || !rows_map(&a.b0, f.wg, f.C, f.F, f.C, 64) ||
      !rows_map(&a.b1, f.wu, f.C, f.F, f.C, 64) || !rows_map(&a.aw, da, f.F, f.T, f.F, 64, 2) ||
      !rows_map(&a.bw, f.x, f.C, f.T, f.x_stride, 64) ||
      !(sx > 1 ? rows_map_f32(&a.out0, parts, f.C, f.T, f.C, sx) : rows_map(&a.out0, f.dx, f.C, f.T, f.dx_stride, 32)) ||
      !(sw > 1 ? rows_map_f32(&a.out1, parts + dx_parts(g), f.C, f.F, f.C, 2 * sw)
               : rows_map(&a.out1, f.dwg, f.C, f.F, f.C, 32)) ||
      !rows_map(&a.out2, f.dwu, f.C, f.F, f.C, 32))
    return cudaErrorInvalidValue;
  e = launch<kSums, kSilu>(a, st);
  return e == cudaSuccess ? join_sums(f, g, parts, st) : e;
}

}  // namespace la
