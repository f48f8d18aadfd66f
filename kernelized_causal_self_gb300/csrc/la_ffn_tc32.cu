// The gated projections in float32 on the tensor cores. A float32 is the sum of three bf16 of 8
// bits each (its top 16 bits, the rounded rest, and the rounded rest of that), so a product
// of two is nine exact products of bf16, of which the three smallest, about 2^-24 of the whole, are
// left out: x y = x0 y0 + x0 y1 + x1 y0 + x1 y1 + x0 y2 + x2 y0, at a sixth of the bf16 rate instead of
// the CUDA cores' thirtieth. An infinity or NaN gives NaN.
//
// The kernels are those of la_ffn_tc.cu (pairs of CTAs, tiles of 256 x 256, the same four products)
// but for three things. A stage holds 64 terms of all three parts of A and of B, so that the six
// products are made from one copy. The tensor cores' sums are taken out every 64 terms (24
// instructions, the largest products last) and added in float32 in registers: their adder cuts
// off what does not fit, always towards zero, which over a long sum would show. And da, du leave as
// their three bf16 parts, which the products behind them read; x and the weights are
// cut up by a kernel before. T 2048, C 512, F 1408: 5 us for that, 49 for da and du, 47 for dx and
// the weights' gradients (750 TFLOP/s of bf16, results 2e-7 off in the 2-norm). T 16384: h in 178 us, 213 with
// a checkpoint; backward 595, 413 from a checkpoint. The 128 sums of a thread take most of its 168
// registers: da and du spill 92 bytes a thread, 140 with silu, the sums behind them 48, h 16.
#include <cuda_bf16.h>

#include "la_ffn_tc.cuh"

namespace la {
namespace {

using namespace ffn;

constexpr int kThreads = 32 * (kWarps + 2);
constexpr int S = 2;
constexpr int kStageBytes = 6 * kTileBytes;  // A's three parts, B's three
constexpr int kSmem = 1024 + S * kStageBytes + kWarps * kStore + 256;

struct Args : Grids {
  CUtensorMap a, b0, b1;         // operands' parts: [3][rows][cols], of da, du [2][3][T][F]
  CUtensorMap aw, bw;            // of dwg and dwu: da, du and x, both read along their rows
  CUtensorMap out0, out1, out2;  // h; the parts of da, du; dx, dwg, dwu. Of cut sums their parts: out0
                                 // [splits][T][C], out1 [2][splits][F][C]
  WorkspaceHeader* hdr;
  signed char* codes;
  unsigned char* exps;
  const float* dh;
  long long dh_stride;
  int clear;
};

template <int KIND, int ACT>
__global__ void __launch_bounds__(kThreads, 1) ffn_tc32_kernel(const __grid_constant__ Args a) {
  constexpr bool DUAL = KIND == kForward || KIND == kGrads;
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
  uint8_t* stages = sm;  // [stage][A0 A1 A2 B0 B1 B2]
  uint8_t* staging = stages + S * kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kWarps * kStore);  // S (the even CTA's count)
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;      // 2: an accumulator holds 64 terms
  uint64_t* acc_empty = acc_full + 2;  // 2 (the even CTA's): both CTAs have read it
  uint64_t* drain = acc_empty + 2;
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
    if (KIND == kSums) {
      prefetch_tensormap(&a.aw);
      prefetch_tensormap(&a.bw);
      prefetch_tensormap(&a.out1);
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
        for (int k = first_step(g, w.split); k < end; ++k) {
          if (!mbar_wait_abort(&empty[s], phase, abort, hdr, kSiteEmpty)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kStageBytes);
          const uint32_t bar = bars + 8 * s;
          const int part = KIND == kSums && !w.dw && k >= g.per ? 1 : 0, kk = (k - part * g.per) * 64;
          const CUtensorMap* mb = w.dw ? &a.bw : (DUAL ? rank != 0 : part != 0) ? &a.b1 : &a.b0;
          uint8_t *ta = stages + s * kStageBytes, *tb = ta + 3 * kTileBytes;
#pragma unroll
          for (int i = 0; i < 3; ++i, ta += kTileBytes, tb += kTileBytes) {
            if constexpr (DUAL) {
              tma_load_3d_pair(ta, &a.a, bar, kk, row, i);
              tma_load_3d_pair(tb, mb, bar, kk, w.n * 128, i);
            } else {
              const int col = w.n * 256 + (int)rank * 128;
              if (!w.dw) {
                tma_load_3d_pair(ta, &a.a, bar, kk, row, part * 3 + i);
              } else {
                tma_load_3d_pair(ta, &a.aw, bar, row, kk, w.part * 3 + i);
                tma_load_3d_pair(ta + kTileBytes / 2, &a.aw, bar, row + 64, kk, w.part * 3 + i);
              }
              tma_load_3d_pair(tb, mb, bar, col, kk, i);
              tma_load_3d_pair(tb + kTileBytes / 2, mb, bar, col + 64, kk, i);
            }
          }
          if (++s == S) s = 0, phase ^= 1;
        }
      }
      // as in la_ffn_tc.cu: the last stages are multiplied, or, if a wait ran out, have landed
      for (uint32_t k = 0; k < S; ++k) {
        const uint32_t turn = k < s ? phase ^ 1 : phase;
        if (ok ? !mbar_wait(&empty[k], turn) : rank == 0 && !mbar_wait(&full[k], turn)) record_timeout(hdr, kSiteDrain);
      }
    }
    __syncwarp();
  } else if (warp == kWarps + 1) {
    // ------------------------------------------------------------------ products
    if (lane == 0 && rank == 0) {
      const uint32_t at = smem_u32(stages);
      const uint64_t da_k = sdesc(at, 16, 1024), da_m = sdesc(at, kTileBytes / 2, 1024);
      const uint64_t db0 = DUAL ? sdesc(at + 3 * kTileBytes, 16, 1024) : sdesc(at + 3 * kTileBytes, kTileBytes / 2, 1024);
      constexpr uint32_t ALONG_K = 32 / 16, ALONG_MN = 2048 / 16, STEP_B = DUAL ? ALONG_K : ALONG_MN, PART = kTileBytes / 16;
      constexpr int ia[6] = {2, 0, 1, 1, 0, 0}, ib[6] = {0, 2, 1, 0, 1, 0};  // the smallest products first
      uint32_t s = 0, phase = 0, n = 0;
      bool ok = true;
      for (int t, i = 0; ok && (t = dealt<KIND>(a, cluster, clusters, i)) >= 0; ++i) {
        int steps = a.g[0].steps, dw = 0;
        if (!DUAL) {
          const Tile w = tile_of<KIND>(a, t);
          dw = w.dw;
          steps = first_step(a.g[dw], w.split + 1) - first_step(a.g[dw], w.split);
        }
        const uint64_t da0 = !DUAL && dw ? da_m : da_k;
        const uint32_t step_a = !DUAL && dw ? ALONG_MN : ALONG_K;
        const uint32_t id = !DUAL && dw ? idesc_bf16(256, 256, true, true) : idesc_bf16(256, 256, false, !DUAL);
        for (int k = 0; k < steps; ++k, ++n) {
          const uint32_t b = n & 1;
          if (n >= 2) ok = mbar_wait_abort(&acc_empty[b], (n / 2 - 1) & 1, abort, hdr, kSiteAccEmpty);
          ok = ok && mbar_wait_abort(&full[s], phase, abort, hdr, kSiteFull);
          if (!ok) break;
          fence_after_sync();
          const uint64_t da = da0 + s * (kStageBytes / 16), db = db0 + s * (kStageBytes / 16);
#pragma unroll
          for (int c = 0; c < 6; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              mma_ss_pair(tbase + 256 * b, da + ia[c] * PART + q * step_a, db + ib[c] * PART + q * STEP_B, id, (c | q) != 0);
          mma_commit_pair(&empty[s]);
          mma_commit_pair(&acc_full[b]);
          if (++s == S) s = 0, phase ^= 1;
        }
      }
      mma_commit_pair_own(drain);
      if (!mbar_wait(drain, 0)) record_timeout(hdr, kSiteDrain);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ results
    uint8_t* st = staging + warp * kStore;
    const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16, half = warp / 4;
    const uint32_t freed = cluster_map(smem_u32(acc_empty), 0);
    auto left = [&]() {  // the last copy out of the staging tile has read it
      if (lane == 0) bulk_wait_read<0>();
      __syncwarp();
    };
    uint32_t n = 0;
    bool ok = true;
    for (int t, i = 0; ok && (t = dealt<KIND>(a, cluster, clusters, i)) >= 0; ++i) {
      const Tile w = tile_of<KIND>(a, t);
      const Grid& g = a.g[w.dw];
      const int row0 = w.m * 256 + (int)rank * 128 + warp % 4 * 32, row = row0 + lane;
      // a thread's 128 sums of its row: 64 columns of a and the same of u, or 128 columns
      float v[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) v[j] = 0.f;
      if (KIND == kGrads && row < g.rows) {  // the thread's piece of dh, into L2 while the sums are made
        const int col = w.n * 128 + 64 * half;
        for (int j = 0; j < 64 && col + j < g.cols; j += 32)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(a.dh + row * a.dh_stride + col + j));
      }
      const int end = first_step(g, w.split + 1);
      for (int k = first_step(g, w.split); k < end; ++k, ++n) {
        const uint32_t b = n & 1;
        if (!mbar_wait_warp(&acc_full[b], n / 2 & 1, abort, hdr, kSiteAccFull)) {
          ok = false;
          break;
        }
        fence_after_sync();
        const uint32_t d = tbase + 256 * b + lanes + (DUAL ? 64 : 128) * half;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[32];
          tmem_ld32(d + (DUAL ? c / 2 * 128 + c % 2 * 32 : c * 32), p);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[c * 32 + j] += __uint_as_float(p[j]);
        }
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(freed + 8 * b);
      }
      if (!ok) break;
      auto leave = [&](const CUtensorMap* to, int col, int mat) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (row0 < g.rows && col < g.cols) tma_store_3d(to, st, col, row0, mat);
          bulk_commit();
        }
      };
      auto leave32 = [&](const float* x, const CUtensorMap* to, int col, int mat) {  // 32 columns in float32
        left();
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<float4*>(st + sw128(lane, e * 16)) = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        leave(to, col, mat);
      };
      const int col0 = w.n * (DUAL ? 128 : 256) + (DUAL ? 64 : 128) * half;
      if constexpr (KIND == kForward) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int f = col0 + c * 32;
          if (a.codes != nullptr) {  // a thread has a block of 32 of a and of u
            const int nb = q8::blocks_of(g.cols);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float* x = v + i * 64 + c * 32;
              float top = fabsf(x[0]);
#pragma unroll
              for (int j = 1; j < 31; j += 2) top = q8::top3(top, x[j], x[j + 1]);
              const uint32_t e = q8::step_of(__float_as_uint(q8::top3(top, x[31], x[31])));
              const float inv = q8::inverse_step(e);
              if (row < g.rows && f < g.cols) {
                const size_t r = 2 * (size_t)row + i;
                signed char* to = a.codes + r * g.cols + f;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (f + j * 8 < g.cols)
                    *reinterpret_cast<uint2*>(to + j * 8) =
                        make_uint2(q8::codes4(x + j * 8, inv, e), q8::codes4(x + j * 8 + 4, inv, e));
                a.exps[r * nb + f / q8::kBlock] = (unsigned char)e;
              }
            }
          }
#pragma unroll
          for (int j = c * 32; j < c * 32 + 32; j += 2) {
            const float2 h = mul2(act2<ACT>(make_float2(v[j], v[j + 1])), make_float2(v[64 + j], v[64 + j + 1]));
            v[j] = h.x, v[j + 1] = h.y;
          }
          leave32(v + c * 32, &a.out0, f, 0);
        }
      } else if constexpr (KIND == kGrads) {
        const float* dh = a.dh + row * a.dh_stride + col0;
        float4 next[4];  // dh, 16 columns at a time, one time ahead
        auto ask = [&](int j0) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            next[i] = row < g.rows && col0 + j0 + 4 * i < g.cols ? __ldg(reinterpret_cast<const float4*>(dh + j0 + 4 * i))
                                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        ask(0);
#pragma unroll
        for (int j0 = 0; j0 < 64; j0 += 16) {  // da and du take the places of a and u
          float d[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) d[4 * i] = next[i].x, d[4 * i + 1] = next[i].y, d[4 * i + 2] = next[i].z, d[4 * i + 3] = next[i].w;
          if (j0 < 48) ask(j0 + 16);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const int j = j0 + i;
            const float2 dv = make_float2(d[i], d[i + 1]);
            float2 f, df;
            act_grad2<ACT>(make_float2(v[j], v[j + 1]), f, df);
            const float2 da = mul2(mul2(dv, make_float2(v[64 + j], v[64 + j + 1])), df), du = mul2(dv, f);
            v[j] = da.x, v[j + 1] = da.y;
            v[64 + j] = du.x, v[64 + j + 1] = du.y;
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            left();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              uint32_t o[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) o[j] = take_part(v[i * 64 + e * 8 + j * 2], v[i * 64 + e * 8 + j * 2 + 1], part);
              *reinterpret_cast<uint4*>(st + sw128(lane, e * 16)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            leave(&a.out0, col0, i * 3 + part);
          }
      } else {
        const bool cut = g.splits > 1;
        const CUtensorMap* to = !w.dw ? &a.out0 : !cut && w.part ? &a.out2 : &a.out1;
#pragma unroll
        for (int c = 0; c < 4; ++c) leave32(v + c * 32, to, col0 + c * 32, cut ? w.part * g.splits + w.split : 0);
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

// The three parts of x's rows (blockIdx.y 0) and of the weights: kEach times 4 neighbours a thread
struct Cut {
  const float *x, *wg, *wu;
  __nv_bfloat16 *px, *pg, *pu;  // [3][rows][C]
  long long T, F, x_stride;
  int C;
};

constexpr int kEach = 4;

__global__ void __launch_bounds__(256) ffn_cut_kernel(const Cut c) {
  const int m = blockIdx.y;
  const float* from = m == 0 ? c.x : m == 1 ? c.wg : c.wu;
  __nv_bfloat16* to = m == 0 ? c.px : m == 1 ? c.pg : c.pu;
  const long long rows = m == 0 ? c.T : c.F, ld = m == 0 ? c.x_stride : c.C;
  const unsigned per = c.C / 4;
  const size_t plane = (size_t)rows * c.C;
  const unsigned long long at = (unsigned long long)blockIdx.x * (256 * kEach);  // (one 64-bit division a CTA)
  const unsigned first = (unsigned)(at % per) + threadIdx.x;
  const long long row0 = (long long)(at / per);
  if (row0 >= rows) return;
  pdl_wait();
  float4 v[kEach];
  long long row[kEach];
  unsigned col[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const unsigned i = first + j * 256;
    row[j] = row0 + i / per;
    col[j] = i % per * 4;
    if (row[j] < rows) v[j] = __ldcs(reinterpret_cast<const float4*>(from + row[j] * ld + col[j]));
  }
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    if (row[j] >= rows) continue;
    __nv_bfloat16* p = to + row[j] * c.C + col[j];
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      const uint32_t lo = take_part(v[j].x, v[j].y, part), hi = take_part(v[j].z, v[j].w, part);
      *reinterpret_cast<uint2*>(p + part * plane) = make_uint2(lo, hi);
    }
  }
}

template <int KIND, int ACT>
cudaError_t launch(Args& a, cudaStream_t st) {
  cudaError_t e = configure_once<ffn_tc32_kernel<KIND, ACT>>(kSmem);
  if (e != cudaSuccess) return e;
  const int tiles = a.g[0].tiles + a.g[1].tiles;
  const int pairs = tiles < sm_count() / 2 ? tiles : sm_count() / 2;
  e = launch_cluster_pdl(ffn_tc32_kernel<KIND, ACT>, dim3(2 * pairs), dim3(kThreads), kSmem, st, 2, a);
  count_launches(1);
  a.clear = 0;
  return e;
}

template <int KIND>
cudaError_t launch_act(Args& a, int act, cudaStream_t st) {
  return act == kSilu   ? launch<KIND, kSilu>(a, st)
         : act == kGelu ? launch<KIND, kGelu>(a, st)
                        : launch<KIND, kGeluTanh>(a, st);
}

// The workspace: header, the parts of x, wg, wu, then (backward) of da, du, and of cut sums
struct Plan {
  size_t w, dact, sums, end;  // offsets in bytes
};

constexpr Costs kCosts{6 * 550, 6000, 1 << 20};  // (parts of any length: sums are taken out every 64 terms)

Plan plan_of(int T, int C, int F, bool backward) {
  Plan p{};
  p.w = kHeaderBytes + align_up(6 * (size_t)T * C, 256);
  p.dact = p.w + align_up(12 * (size_t)F * C, 256);
  p.end = p.dact;
  if (!backward) return p;
  const Grids& g = sums_grids(T, C, F, kCosts);
  p.sums = p.dact + align_up(12 * (size_t)T * F, 256);
  p.end = p.sums + sizeof(float) * (dx_parts(g) + dw_parts(g));
  return p;
}

struct Parts {
  __nv_bfloat16 *x, *wg, *wu;
};

cudaError_t cut(const FfnGate& f, char* ws, const Plan& p, Parts& to, cudaStream_t st) {
  to.x = reinterpret_cast<__nv_bfloat16*>(ws + kHeaderBytes);
  to.wg = reinterpret_cast<__nv_bfloat16*>(ws + p.w);
  to.wu = to.wg + 3 * (size_t)f.F * f.C;
  const Cut c{static_cast<const float*>(f.x), static_cast<const float*>(f.wg), static_cast<const float*>(f.wu),
              to.x, to.wg, to.wu, f.T, f.F, f.x_stride, f.C};
  const long long most = (long long)(f.T > f.F ? f.T : f.F) * (f.C / 4);  // (T <= 2^24, C <= 2^16: an int of CTAs)
  const cudaError_t e = launch_pdl(ffn_cut_kernel, dim3((unsigned)((most + 256 * kEach - 1) / (256 * kEach)), 3), dim3(256), 0, st, c);
  count_launches(1);
  return e;
}

// a = x wg^T, u = x wu^T
bool products(Args& a, const FfnGate& f, const Parts& p) {
  static_cast<Grids&>(a) = products_grid(f.T, f.C, f.F);
  a.clear = 1;
  return rows_map(&a.a, p.x, f.C, f.T, f.C, 128, 3) && rows_map(&a.b0, p.wg, f.C, f.F, f.C, 128, 3) &&
         rows_map(&a.b1, p.wu, f.C, f.F, f.C, 128, 3);
}

}  // namespace

size_t ffn_tc32_workspace(int T, int C, int F, bool backward) { return plan_of(T, C, F, backward).end; }

cudaError_t ffn_tc32_forward(const FfnGate& f, void* ws, cudaStream_t st) {
  Parts p;
  cudaError_t e = cut(f, static_cast<char*>(ws), plan_of(f.T, f.C, f.F, false), p, st);
  if (e != cudaSuccess) return e;
  Args a{};
  a.hdr = static_cast<WorkspaceHeader*>(ws);
  a.codes = f.codes;
  a.exps = f.exps;
  if (!products(a, f, p) || !rows_map_f32(&a.out0, f.h, f.F, f.T, f.h_stride)) return cudaErrorInvalidValue;
  return launch_act<kForward>(a, f.act, st);
}

cudaError_t ffn_tc32_backward(const FfnGate& f, void* ws, cudaStream_t st) {
  const Plan plan = plan_of(f.T, f.C, f.F, true);
  char* at = static_cast<char*>(ws);
  __nv_bfloat16* dact = reinterpret_cast<__nv_bfloat16*>(at + plan.dact);  // [da, du][3][T][F]
  float* parts = reinterpret_cast<float*>(at + plan.sums);
  Parts p;
  cudaError_t e = cut(f, at, plan, p, st);
  if (e != cudaSuccess) return e;
  Args a{};
  a.hdr = static_cast<WorkspaceHeader*>(ws);
  if (f.codes != nullptr || ffn_few(f.T, f.F, f.dtype)) {
    e = f.codes != nullptr ? ffn_kept_grads(f, dact, st) : ffn_few_grads(f, dact, st);
    a.clear = 1;
  } else {
    a.dh = static_cast<const float*>(f.dh);
    a.dh_stride = f.dh_stride;
    if (!products(a, f, p) || !rows_map(&a.out0, dact, f.F, f.T, f.F, 32, 6)) return cudaErrorInvalidValue;
    e = launch_act<kGrads>(a, f.act, st);
  }
  if (e != cudaSuccess) return e;

  const Grids& g = sums_grids(f.T, f.C, f.F, kCosts);
  static_cast<Grids&>(a) = g;
  const int sx = g.g[0].splits, sw = g.g[1].splits;
  if (!rows_map(&a.a, dact, f.F, f.T, f.F, 128, 6) || !rows_map(&a.b0, p.wg, f.C, f.F, f.C, 64, 3) ||
      !rows_map(&a.b1, p.wu, f.C, f.F, f.C, 64, 3) || !rows_map(&a.aw, dact, f.F, f.T, f.F, 64, 6) ||
      !rows_map(&a.bw, p.x, f.C, f.T, f.C, 64, 3) ||
      !(sx > 1 ? rows_map_f32(&a.out0, parts, f.C, f.T, f.C, sx) : rows_map_f32(&a.out0, f.dx, f.C, f.T, f.dx_stride)) ||
      !(sw > 1 ? rows_map_f32(&a.out1, parts + dx_parts(g), f.C, f.F, f.C, 2 * sw)
               : rows_map_f32(&a.out1, f.dwg, f.C, f.F, f.C)) ||
      !rows_map_f32(&a.out2, f.dwu, f.C, f.F, f.C))
    return cudaErrorInvalidValue;
  e = launch<kSums, kSilu>(a, st);
  return e == cudaSuccess ? join_sums(f, g, parts, st) : e;
}

}  // namespace la
