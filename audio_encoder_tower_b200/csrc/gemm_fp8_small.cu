// The block-scaled e4m3 product (gemm_fp8.cu) for few rows of A, where the time is that of
// reading W once and of the launch.
//
// The operands change places: 128 rows of W are the MMA's M and a tile of 16 to 64 rows of A
// its N, so that a single row of A does not pay for a tile of 256. K is split over the CTAs of
// a cluster, so that a narrow layer still has enough SMs reading. Row m of a tile is added up
// and written by CTA m % split: every CTA sends its fp32 partial sums there with one bulk copy
// per CTA (loads over the cluster took 5 to 10 us, stores 1 to 3), and they are added in rank
// order, so a call always gives the same bits.
// One tile per CTA, run once from start to end, so code size counts as well: an unrolled
// epilogue spent most of its time fetching instructions. The loads start before the rest of
// the set-up.
//   warp 0  TMA producer;  warp 1  MMA issuer;  warp 2  scales;  then all of them  epilogue
#include <math.h>

#include "fp8.cuh"
#include "internal.h"

namespace enc {

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // 2 s: far above any legitimate wait
constexpr uint32_t kWBytes = 128 * kBK;
constexpr int kScaleSlots = 4, kScaleTmemSlots = 2;                       // in shared memory, in TMEM
constexpr uint32_t kScaleSlotBytes = 2 * 512;                             // 128 rows of W, up to 64 of A
constexpr uint32_t kTmemCols = 256, kScaleCol = 128, kScaleSlotCols = 8;  // accumulator from column 0

// Two CTAs per SM.
// The epilogue takes a row per warp, one after another: the higher the tile, the more warps
// (64 x 4192 x 192, tiles of 32 rows: 4.5 us with four warps, 3.9 with eight; 113 x 3568 x 1280,
// of 64 rows: 6.9 with eight, 6.5 with sixteen). A call of up to 16 rows starts sooner with four.
template <int BT>
struct Cfg {
  static constexpr int kStages = BT == 16 ? 5 : BT == 64 ? 3 : 4;
  static constexpr int kThreads = BT == 16 ? 128 : BT == 32 ? 256 : 512;
  static constexpr uint32_t kABytes = BT * kBK;
  static constexpr uint32_t kStageBytes = kWBytes + kABytes;
  static constexpr size_t kSmem = 1024 + kStages * (size_t)kStageBytes + BT * 512 /*partial sums*/ +
                                  kScaleSlots * kScaleSlotBytes + 256 /*barriers*/;
  static_assert(kStages * kStageBytes >= BT * 512, "outgoing partial sums reuse the ring");
};

__device__ __forceinline__ void umma_mxf8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::
          "r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Shared memory of this CTA to that of another of the cluster, counted on its barrier.
__device__ __forceinline__ void bulk_copy_cluster(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :
               : "r"(dst), "r"(smem_u32(src)), "r"(bytes), "r"(bar)
               : "memory");
}

template <int BT>
__global__ void __launch_bounds__(Cfg<BT>::kThreads)
gemm_fp8_small_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                      const GemmFp8Params p, void* out, int out_kind, int split) {
  using C = Cfg<BT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sW = smem;
  uint8_t* sA = sW + C::kStages * kWBytes;
  float* outgoing = reinterpret_cast<float*>(smem);                           // [owner][its rows][128], after the MMAs
  float* incoming = reinterpret_cast<float*>(sA + C::kStages * C::kABytes);   // [rank][this CTA's rows][128]
  uint8_t* sS = reinterpret_cast<uint8_t*>(incoming) + BT * 512;
  uint64_t* full = reinterpret_cast<uint64_t*>(sS + kScaleSlots * kScaleSlotBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* sfull = empty + C::kStages;
  uint64_t* sempty = sfull + kScaleSlots;
  uint64_t* done = sempty + kScaleSlots;
  uint64_t* received = done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(received + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x) % split, tile = static_cast<int>(blockIdx.x) / split;
  const int tiles_n = (p.N + 127) / 128;
  const int n0 = (tile % tiles_n) * 128, m0 = (tile / tiles_n) * BT;
  const int kb0 = static_cast<int>((int64_t)p.num_kb * rank / split);
  const int kb1 = static_cast<int>((int64_t)p.num_kb * (rank + 1) / split);

  const int rows = min(BT, p.M - m0);                  // of this tile
  const int log = 31 - __clz(split), per = BT >> log;  // rows a CTA may own
  const int mine = (rows - rank + split - 1) >> log;   // and does own

  uint32_t armed = 0, armed_phase = 0;   // producer lane: as in the 256 x 256 kernel
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int s = 0; s < kScaleSlots; ++s) { mbar_init(&sfull[s], 1); mbar_init(&sempty[s], 1); }
    mbar_init(done, 1);
    mbar_init(received, 1);
    *abort_flag = 0;
    fence_barrier_init();
    if (split > 1 && mine > 0) mbar_arrive_expect_tx(received, static_cast<uint32_t>(split * mine * 512));
  }
  __syncwarp();
  // Warp 0 has set the barriers up and goes on to the loads; the others wait for it and for
  // TMEM, which it needs only after `done`. Nothing is sent to another CTA's shared memory
  // before the wait that matches this arrival.
  if (split > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  uint32_t tmem_base = 0;
  if (warp == 0) {
    asm volatile("bar.arrive 1, %0;" ::"n"(C::kThreads) : "memory");
  } else {
    if (warp == 1) { tmem_alloc(tmem_slot, kTmemCols); tmem_relinquish(); }
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(C::kThreads) : "memory");
    tc_fence_after();
    tmem_base = *tmem_slot;
  }
  volatile int* abort_v = abort_flag;
  grid_dependency();   // global memory from here on

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
#pragma unroll 1
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_v, kWaitLimitNs)) { ok = false; break; }
        mbar_arrive_expect_tx(&full[stage], C::kStageBytes);
        tma_load_2d(sW + stage * kWBytes, &map_w, &full[stage], kb * kBK, n0);
        tma_load_2d(sA + stage * C::kABytes, &map_a, &full[stage], kb * kBK, m0);
        armed |= 1u << stage;
        armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) { set_status(p.status, kDevTimeout); *abort_v = 1; }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    const uint64_t wdesc0 = smem_desc_sw128(smem_u32(sW)), adesc0 = smem_desc_sw128(smem_u32(sA));
    int stage = 0, slot = 0;
    uint32_t phase = 0, sphase = 0;
    bool ok = true, wrapped = false;   // groups before the third have no earlier user of their TMEM columns
#pragma unroll 1
    for (int kb = kb0; kb < kb1; ++kb) {
      const uint32_t id = kb & 3;
      const bool first = kb == kb0 || id == 0, last = id == 3 || kb + 1 == kb1;
      const uint32_t sfw = tmem_base + kScaleCol + (slot & (kScaleTmemSlots - 1)) * kScaleSlotCols, sfa = sfw + 4;
      if (first) {
        const int before = (slot + kScaleSlots - kScaleTmemSlots) & (kScaleSlots - 1);
        if (!mbar_wait_warp(&sfull[slot], sphase, abort_v, kWaitLimitNs) ||
            ((wrapped || slot >= kScaleTmemSlots) &&
             !mbar_wait_warp(&sempty[before], sphase ^ (slot < kScaleTmemSlots ? 1u : 0u), abort_v, kWaitLimitNs))) {
          ok = false;
          break;
        }
      }
      if (!mbar_wait_warp(&full[stage], phase, abort_v, kWaitLimitNs)) { ok = false; break; }
      tc_fence_after();
      const uint64_t wdesc = wdesc0 + static_cast<uint64_t>(stage) * (kWBytes >> 4);
      const uint64_t adesc = adesc0 + static_cast<uint64_t>(stage) * (C::kABytes >> 4);
      if (elect_one()) {
        if (first) {
          const uint64_t sdesc = smem_desc_scales(smem_u32(sS + slot * kScaleSlotBytes));
          tmem_cp_scales(sfw, sdesc);
          tmem_cp_scales(sfa, sdesc + (512 >> 4));
        }
#pragma unroll
        for (int k = 0; k < kBK / 32; ++k)
          umma_mxf8(tmem_base, wdesc + static_cast<uint64_t>(2 * k), adesc + static_cast<uint64_t>(2 * k),
                    idesc_mxf8(128, BT) | idesc_scale_id(id), sfw, sfa, (kb != kb0 || k != 0) ? 1u : 0u);
        umma_commit(&empty[stage]);
        if (last) umma_commit(&sempty[slot]);
      }
      __syncwarp();
      if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
      if (last && ++slot == kScaleSlots) { slot = 0; sphase ^= 1u; wrapped = true; }
    }
    if (!ok && lane == 0) { set_status(p.status, kDevTimeout); *abort_v = 1; }
    if (elect_one()) umma_commit(done);   // every MMA issued so far
    __syncwarp();
  } else if (warp == 2) {
    // -------------------------------------------------------------- scales
    int slot = 0;
    uint32_t sphase = 0;
    bool ok = true;
#pragma unroll 1
    for (int g = kb0 >> 2; g < (kb1 + 3) >> 2; ++g) {
      uint32_t w[8];
#pragma unroll
      for (int c = 0; c < 4; ++c) w[c] = scale_word(p.w_scales, p.k_pitch, n0 + 32 * c + lane, p.N, g);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        w[4 + c] = c * 32 < BT ? scale_word(p.a_scales, p.k_pitch, m0 + 32 * c + lane, p.M, g) : kUnitScale;
      if (!mbar_wait_warp(&sempty[slot], sphase ^ 1u, abort_v, kWaitLimitNs)) { ok = false; break; }
      uint4* dst = reinterpret_cast<uint4*>(sS + slot * kScaleSlotBytes) + lane;
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[32] = make_uint4(w[4], w[5], w[6], w[7]);
      fence_proxy_async_smem();   // tcgen05.cp reads them through the async proxy
      __syncwarp();
      if (lane == 0) mbar_arrive(&sfull[slot]);
      if (++slot == kScaleSlots) { slot = 0; sphase ^= 1u; }
    }
    if (!ok && lane == 0) { set_status(p.status, kDevTimeout); *abort_v = 1; }
  }
  __syncwarp();

  // -------------------------------------------------------------- epilogue
  const int n = n0 + 4 * lane;   // columns n .. n + 3 from here on (N is a multiple of 16)
  float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.bias && n < p.N) bias = __ldg(reinterpret_cast<const float4*>(p.bias + n));
  // The MMA warp commits `done` even when it gave up.
  if (!mbar_wait_warp(done, 0, nullptr, kWaitLimitNs) && lane == 0) set_status(p.status, kDevTimeout);
  __syncthreads();
  tc_fence_after();
  tmem_base = *tmem_slot;
  // accumulators (lane = column of the output) to shared memory, by owner; rows past the tile's
  // last valid one go along up to the next multiple of 16
#pragma unroll 1
  for (int m = warp / 4 * 16; m < rows; m += C::kThreads / 8) {
    uint32_t v[16];
    tmem_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(warp % 4 * 32) << 16) + m, v);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i)
      outgoing[(((m + i) & (split - 1)) * per + ((m + i) >> log)) * 128 + threadIdx.x % 128] = __uint_as_float(v[i]);
  }
  const float* sums = outgoing;
  if (split > 1) {
    fence_proxy_async_smem();
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 0 && lane < split) {
      const int theirs = (rows - lane + split - 1) >> log;
      if (theirs > 0)
        bulk_copy_cluster(peer_addr(incoming + rank * theirs * 128, lane), outgoing + lane * per * 128,
                          static_cast<uint32_t>(theirs * 512), peer_addr(received, lane));
    }
    __syncwarp();
    if (mine > 0 && !mbar_wait_warp(received, 0, nullptr, kWaitLimitNs) && lane == 0)
      set_status(p.status, kDevTimeout);
    __syncwarp();
    // every copy to this CTA has arrived; when all have said so, every CTA's own have been read
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    sums = incoming;
  } else {
    __syncthreads();
  }
  const int stride = split > 1 ? mine * 128 : per * 128;   // from one rank's sums to the next
#pragma unroll 1
  for (int j = warp; j < mine; j += C::kThreads / 32) {   // one row per warp
    const float4* s4 = reinterpret_cast<const float4*>(sums + j * 128) + lane;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (BT > 16 && split == 1) {
      y = s4[0];
    } else {
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < split) {
          const float4 t = s4[r * stride / 4];
          y = make_float4(y.x + t.x, y.y + t.y, y.z + t.z, y.w + t.w);
        }
    }
    y = make_float4(y.x + bias.x, y.y + bias.y, y.z + bias.z, y.w + bias.w);
    const int64_t m = m0 + rank + ((int64_t)j << log), at = m * p.N + n;
    const float4 sum = y;
    if (p.gelu) {   // the form for fp32 whatever the output: rows are few
      gelu_fp32_2(y.x, y.y);
      gelu_fp32_2(y.z, y.w);
    }
    if (out_kind == ENC_FP8_OUT_FP8) {
      // the warp has a whole block of 128 columns (zeros past N)
      uint32_t top = max(max(finite_abs_bits(y.x), finite_abs_bits(y.y)),
                         max(finite_abs_bits(y.z), finite_abs_bits(y.w)));
      const uint32_t byte = e8m0_of_amax(__reduce_max_sync(0xffffffffu, top));
      const float inv = e8m0_inverse(byte);
      if (n < p.N)   // the products with zero turn an infinite sum into NaN, of which GELU may have made a zero
        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(out) + at) =
            e4m3x4(fmaf(sum.x, 0.f, y.x * inv), fmaf(sum.y, 0.f, y.y * inv), fmaf(sum.z, 0.f, y.z * inv),
                   fmaf(sum.w, 0.f, y.w * inv));
      const int g = n0 / kFp8Block + lane;   // the block's scale, and after the row's last block the padding
      if (lane == 0 || (n0 + kFp8Block >= p.N && g < p.out_pitch))
        p.out_scales[m * p.out_pitch + g] = static_cast<uint8_t>(lane == 0 ? byte : 127u);
    } else if (n < p.N) {
      if (out_kind == ENC_FP8_OUT_BF16) {
        *reinterpret_cast<uint2*>(reinterpret_cast<bf16*>(out) + at) =
            make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
      } else {
        float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + at);
        if (out_kind == ENC_FP8_OUT_RESID) {
          const float4 t = *o;
          y = make_float4(y.x + t.x, y.y + t.y, y.z + t.z, y.w + t.w);
        }
        *o = y;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0 && lane == 0 && *abort_v) {
    for (int s = 0; s < C::kStages; ++s)
      if (armed & (1u << s)) mbar_wait(&full[s], (armed_phase >> s) & 1u, nullptr, kWaitLimitNs / 4);
  }
  __syncwarp();
  if (split > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <int BT>
cudaError_t launch_bt(const CUtensorMap& map_a, const CUtensorMap& map_w, int split, const GemmFp8Params& p, void* out,
                      int out_kind, cudaStream_t stream) {
  static DeviceOnce once;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidValue;
  if (!once.run(dev, [] {
        return cudaFuncSetAttribute(gemm_fp8_small_kernel<BT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)Cfg<BT>::kSmem) == cudaSuccess;
      }))
    return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(((p.N + 127) / 128) * ((p.M + BT - 1) / BT) * split);
  return launch_overlapped(gemm_fp8_small_kernel<BT>, grid, Cfg<BT>::kThreads, Cfg<BT>::kSmem, split, stream, map_a, map_w, p,
                           out, out_kind, split);
}

}  // namespace

GemmFp8SmallPlan plan_gemm_fp8_small(int M, int N, int K, int sm_count) {
  // The time of this kernel and of the 256 x 256 one estimated (us), and the least taken. The
  // coefficients are fitted to 700 shapes, M 1 to 3000, N 64 to 5200, K 100 to 6500: the choice
  // is within 1% of the best one on the average. Per CTA: the blocks of K one after another, the
  // tile's epilogue, with K split the exchange of the sums (both go with the tile's height), and
  // what all the CTAs' loads cost each other. From about one CTA per SM on (somewhat fewer where
  // clusters of 4 or 8 do not come out even in a GPC) some share an SM, which pays where each has
  // a long way to go. Examples (this kernel / the other):
  //   1 x 5120 x 1280  4.0 / 8.7    64 x 1280 x 1280   4.3 / 6.6    128 x 3840 x 1024  5.3 / 6.8
  //   1 x 1280 x 5120  4.1 / 13.3   400 x 1280 x 1280  6.1 / 7.2    400 x 1280 x 5120  11.8 / 14.6
  const int kb = fp8_blocks(K);
  const int64_t columns = (N + 127) / 128, pair_tiles = (int64_t)((M + 255) / 256) * ((N + 255) / 256);
  GemmFp8SmallPlan plan = {0, 0};
  float least;
  if (M <= 32) {   // at any width, for the other kernel would compute 256 rows (32 x 16384 x 1280 7.7 / 10.5)
    plan = {M <= 16 ? 16 : 32, 1};
    least = INFINITY;
  } else if (2 * pair_tiles <= sm_count) {   // a pair of SMs per tile or per half of one
    const bool halves = 4 * pair_tiles <= sm_count;
    least = 3.9f + 0.235f * kb + (halves ? 0.f : 2.45f) + 0.0029f * (halves ? 2 * pair_tiles : pair_tiles) * kb;
  } else {
    return plan;
  }
  for (int tile_m = 16; tile_m <= 64; tile_m *= 2)
    for (int split = 1; split <= 8 && split <= kb; split *= 2) {
      const int64_t ctas = columns * ((M + tile_m - 1) / tile_m) * split;
      const int64_t over = ctas - sm_count + (split < 4 ? 0 : split == 4 ? 12 : 20);
      if (ctas > 2 * sm_count) break;
      const int depth = (kb + split - 1) / split;
      const float t = 2.0f + 0.26f * depth + 0.012f * tile_m + (split > 1 ? 0.015f * tile_m : 0.f) +
                      (split > 4 ? 0.2f : 0.f) + 2e-5f * ctas * depth * tile_m +
                      (over > 0 ? 1.f + 0.2f * depth * over / sm_count : 0.f);
      if (t < least) {
        plan = {tile_m, split};
        least = t;
      }
    }
  return plan;
}

cudaError_t launch_gemm_fp8_small(const CUtensorMap& map_a, const CUtensorMap& map_w, const GemmFp8SmallPlan& plan,
                                  const GemmFp8Params& p, void* out, int out_kind, cudaStream_t stream) {
  if (p.M <= 0) return cudaSuccess;
  switch (plan.tile_m) {
    case 16: return launch_bt<16>(map_a, map_w, plan.split, p, out, out_kind, stream);
    case 32: return launch_bt<32>(map_a, map_w, plan.split, p, out, out_kind, stream);
    case 64: return launch_bt<64>(map_a, map_w, plan.split, p, out, out_kind, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace enc
