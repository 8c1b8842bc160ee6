// tcgen05 GEMM on e4m3 operands with a power-of-two scale for each block of 128
// elements along K, fp32 accumulation in TMEM, fused epilogues:
//
//   out[M, N] = act(sum_kb 2^(ea[m, kb] + ew[n, kb]) sum_{k in kb} A[m, k] W[n, k] + bias[n])
//
// The tensor cores apply the scales themselves (kind::mxf8f6f4, one e8m0 scale per
// row and 32 elements of K): the block's scale is used by the four MMAs of K = 32
// that make up a block, so the accumulator needs no correction between blocks.
//
// Where the scales live. The MMA reads them from TMEM: lane l, column c of a
// four-column group holds, in four bytes, the scales of row 32 c + l, repeated in
// all four lane quarters; the instruction descriptor picks the byte. Four
// consecutive blocks of a row are one 32-bit word of the caller's scale matrix,
// so one word per row serves K = 512 and the byte index is the block modulo four.
// A warp gathers the words into shared memory (16 bytes per lane: rows l, l + 32,
// l + 64, l + 96) and the MMA thread copies them to TMEM with tcgen05.cp.
#include <cudaTypedefs.h>

#include "fp8.cuh"
#include "internal.h"

namespace enc {

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // 2 s: far above any legitimate wait

// D[tmem of both CTAs] (+)= (A * scales) (B * scales)^T, M = 256 over the pair.
__device__ __forceinline__ void umma_mxf8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::
          "r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// 32 rows of 16 bytes of shared memory (512 contiguous bytes) to four TMEM columns,
// repeated in the four lane quarters; each CTA of the pair copies its own.
__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// Whether the phase of `bar` with the given parity is complete, without waiting.
__device__ __forceinline__ bool mbar_peek(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void st_cluster_v4(uint32_t cluster_addr, const uint4& v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// --------------------------------------------------------------- shape of the kernel
// A cluster of two CTAs computes 256 x 256 tiles (M = 256 over the pair). CTA r holds
// rows 128 r .. of the A tile and half of the W tile's rows in a ring of 32 KB stages.
//   warp 0   TMA producer;  warp 1  (first CTA) MMA issuer
//   warps 2, 3  (first CTA) scales of both CTAs, the second's by stores over the cluster. The
//            issuer's tcgen05.cp reads them in the other CTA's shared memory, so they are handed
//            over at cluster scope: a proxy fence of every lane, an arrival that releases and a wait
//            that acquires, on a barrier of the first CTA. Fence and release take about 900 and 1,200
//            cycles, a group of four blocks 1,000 to 2,000: two warps in turn and four slots hide
//            that but for a unit's first group. (A fence.acq_rel.cluster of every lane before the
//            release: 24000 x 1280 x 5120 123 -> 134 us; instead of the release 124. An arrival
//            from the second CTA would pay for the release as well.)
//   warps 4..  epilogue: warps of a TMEM lane quarter split the tile's columns
// TMEM has 512 columns: two accumulators of 256 and the scales do not fit side by side.
// The accumulators overlap instead, by 32 columns: 0..255 and 224..479, scales from
// 480. The half of a tile that shares them with the tile before may start once the epilogue
// has read them there, which it therefore does first. Until then the MMAs of the tile's other
// half run, over the first kEarly blocks of K (as N = 128 each; from there on N = 256), so that
// the tensor cores do not wait for the epilogue between tiles.
// Measured (one B200, 20 launches in a replayed graph): 24000 x 5120 x 1280 with GELU to e4m3 136 to
// 137 us (2,300 TFLOP/s), 18737 x 3840 x 1280 to bf16 82 us, 24000 x 1280 x 5120 to fp32 124 us (2,540).
// Called for longer the clock falls: 164 to 166 us and 98 to 99. Power bounds these: the SM clock is
// 1.46 GHz with the tensor pipe busy 63% of the cycles at K = 1280 and 1.25 GHz with 86% at 5120.
// Added to fp32 (24000 x 1280 x 1280) 59 us: plain fp32 stores of that shape take 45, HBM is 60% busy;
// the difference is the reductions in L2.
// Smaller grids are bound by an SM's intake from L2, about 58 bytes a cycle: 32 KB per 512 cycles of
// MMAs for a full unit.
constexpr int kEpiWarp0 = 4;
constexpr int kStages = 5;
constexpr int kEarly = 2;   // < kStages, < 4 (one group of scales). fc1: 0 blocks 140.5 us, 2 137.2, 3 138 to 140
constexpr uint32_t kOperandBytes = 128 * kBK;          // per stage: this CTA's 128 rows of A, and of W
constexpr uint32_t kTmemCols = 512, kAcc1 = 224, kScaleCol = 480, kScaleSlotCols = 12;
constexpr uint32_t kScaleSlotBytes = 3 * 512;          // A: 128 rows, W: 256 rows
constexpr int kScaleSlots = 4, kScaleTmemSlots = 2;    // in shared memory, in TMEM

constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr size_t kSmemBytes = 1024 + kStages * (size_t)(2 * kOperandBytes) + kEpiWarps * 4096 /*staging*/ +
                              kScaleSlots * kScaleSlotBytes + kEpiWarps * 512 /*bias*/ + 2048 /*amax*/ + 512;

// Work units: tiles of 256 x 256 in row-major order, the last `tail` of them as two
// halves of 128 columns, so that a last wave under half full keeps more SMs busy. A last
// column tile of at most 128 columns is one narrow unit. An element's K order is the
// same in each.
struct Unit {
  int m0, n0, width;
};
__device__ __forceinline__ Unit unit_at(const GemmFp8Params& p, int u) {
  const int nfull = p.num_tiles - p.tail;
  const int h = u - nfull, tile = h < 0 ? u : nfull + (h >> 1);
  Unit t{(tile / p.tiles_n) * 256, (tile % p.tiles_n) * 256, 256};
  if (h >= 0) { t.n0 += (h & 1) * 128; t.width = 128; }
  if (p.N - t.n0 <= 128) t.width = 128;   // also where n0 >= N: such a half loads zeros and stores nothing
  return t;
}

// Four values from the warp's copy of the bias (all lanes the same address: a broadcast).
__device__ __forceinline__ float4 lds4(const float* p) { return *reinterpret_cast<const float4*>(p); }

template <bool kGelu, bool kE4m3, int n>
__device__ __forceinline__ void bias_act(float (&t)[n], const float* bias) {
#pragma unroll
  for (int k = 0; k < n; k += 4) {
    const float4 b = lds4(bias + k);
    add2(t[k], t[k + 1], t[k], t[k + 1], b.x, b.y);
    add2(t[k + 2], t[k + 3], t[k + 2], t[k + 3], b.z, b.w);
    if constexpr (kGelu && kE4m3) {
      gelu_e4m3_2(t[k], t[k + 1]);
      gelu_e4m3_2(t[k + 2], t[k + 3]);
    } else if constexpr (kGelu) {
      gelu_bf16_2(t[k], t[k + 1]);
      gelu_bf16_2(t[k + 2], t[k + 3]);
    }
  }
}

// Where the two warps of a narrow unit meet that hold the halves of the same rows' block of 128
// columns: each writes its amax and reads the other's after a barrier of the two. The buffer
// alternates with the accumulator, so a warp may be one unit ahead of the other. (An mbarrier in
// place of the hardware barrier makes the full unit's path spill: fc1 139 -> 156 us.)
struct Halves {
  uint32_t* amax;   // [2][128] of this unit
  int half, row, barrier;
  __device__ __forceinline__ void meet() const { asm volatile("bar.sync %0, 64;" ::"r"(barrier) : "memory"); }
  __device__ __forceinline__ uint32_t join(uint32_t v) const {
    amax[half * 128 + row] = v;
    meet();
    return max(v, amax[(half ^ 1) * 128 + row]);
  }
};

// e4m3 epilogue of 32 rows by one warp: a block of 128 columns from n0 (n = 128), or this warp's
// half of it (n = 64; n0 is the block's first column in both, taddr and bias the half's).
// The thread's part of the row stays in registers until the block's scale is known. (Half a block
// in each of 16 warps on full units as well keeps up with the MMAs where this is the slower side,
// but 24000 x 5120 x 1280 with GELU took 156 us so against 147 then: the chip is at its power limit,
// and that form does more work. On narrow units the halves occupy warps that would be idle.)
template <int n, bool kGelu, typename Release, typename Done>
__device__ __forceinline__ void epilogue_e4m3(const GemmFp8Params& p, const CUtensorMap* map_c, int r0, int n0,
                                              uint32_t taddr, uint8_t* stage, const float* bias, const Halves& halves,
                                              int lane, Release&& release, Done&& done) {
  float v[n];
#pragma unroll
  for (int c = 0; c < n; c += 32) tmem_ld_32x32b_x32(taddr + c, *reinterpret_cast<uint32_t(*)[32]>(&v[c]));
  if (lane == 0) bulk_wait_read0();
  tmem_wait_ld();
  release();
  done();
  __syncwarp();   // the previous store has read the staging tile
  bias_act<kGelu, true>(v, bias);
  float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < n; j += 8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) top[k] = fmaxf(fmaxf(top[k], fabsf(v[j + 2 * k])), fabsf(v[j + 2 * k + 1]));
  }
  uint32_t bits = __float_as_uint(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));   // passes over NaN
  if constexpr (n == 64) bits = halves.join(bits);
  // an infinity in a row: the largest finite magnitude instead (both halves' warps see the same)
  if (__any_sync(0xffffffffu, bits >= 0x7F800000u)) {
    bits = 0;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      bits = max(bits, finite_abs_bits(v[j]));
      v[j] = fmaf(v[j], 0.f, v[j]);       // and the infinity turns into NaN
    }
    if constexpr (n == 64) {
      halves.meet();                      // both have read what the other wrote
      bits = halves.join(bits);
    }
  }
  const uint32_t byte = e8m0_of_amax(bits);
  const float inv = e8m0_inverse(byte);
  const int piece0 = n == 64 ? 4 * halves.half : 0;   // of the row's eight 16-byte pieces
  uint4* row = reinterpret_cast<uint4*>(stage + lane * 128);
#pragma unroll
  for (int j = 0; j < n / 16; ++j) {
    float t[16];
#pragma unroll
    for (int k = 0; k < 16; k += 2) mul2(t[k], t[k + 1], v[16 * j + k], v[16 * j + k + 1], inv, inv);
    row[(piece0 + j) ^ (lane & 7)] = make_uint4(e4m3x4(t[0], t[1], t[2], t[3]), e4m3x4(t[4], t[5], t[6], t[7]),
                                                e4m3x4(t[8], t[9], t[10], t[11]), e4m3x4(t[12], t[13], t[14], t[15]));
  }
  fence_proxy_async_smem();
  if constexpr (n == 64) halves.meet();
  else __syncwarp();
  if (n == 64 && halves.half) return;
  if (lane == 0) {
    tma_store_2d(map_c, stage, n0, r0);
    bulk_commit();
  }
  const int r = r0 + lane, g = n0 / kFp8Block;
  if (r < p.M) {
    uint8_t* s = p.out_scales + (int64_t)r * p.out_pitch + g;
    *s = static_cast<uint8_t>(byte);
    if (g + 1 == fp8_blocks(p.N))
      for (int i = g + 1; i < p.out_pitch; ++i) *++s = 127;
  }
}

// Epilogue of 32 rows x `cols` columns (from output column n0) by one warp. `bias`: the
// warp's copy of those columns' bias in shared memory, zeros where there is none. `release`
// is called once, as soon as the columns shared with the other accumulator have been read, and
// `done` when all have been. Chunks run upwards or, with `down`, downwards, so that those come first.
template <int kEpi, bool kGelu, typename Release, typename Done>
__device__ __forceinline__ void epilogue(const GemmFp8Params& p, const CUtensorMap* map_c, int r0, int n0, int cols,
                                         uint32_t taddr, bool down, uint8_t* stage, const float* bias, int lane,
                                         Release&& release, Done&& done) {
  constexpr int kChunk = kEpi == ENC_FP8_OUT_BF16 ? 64 : 32;   // 128 bytes of a row
  const int nc = cols / kChunk;
#pragma unroll 1
  for (int i = 0; i < nc; ++i) {
    const int c = (down ? nc - 1 - i : i) * kChunk;
    if (n0 + c >= p.N) continue;
    float v[kChunk];
#pragma unroll
    for (int j = 0; j < kChunk; j += 32)
      tmem_ld_32x32b_x32(taddr + c + j, *reinterpret_cast<uint32_t(*)[32]>(&v[j]));
    if (lane == 0) bulk_wait_read0();   // the previous store has read the staging tile
    tmem_wait_ld();
    if (i == 0) release();
    if (i + 1 == nc) done();
    __syncwarp();
    if constexpr (kEpi == ENC_FP8_OUT_BF16) {
      bias_act<kGelu, false>(v, bias + c);
    } else {
      bias_act<false, false>(v, bias + c);
      if constexpr (kGelu) {   // fp32 keeps what the shorter form would lose
#pragma unroll
        for (int k = 0; k < kChunk; k += 2) gelu_fp32_2(v[k], v[k + 1]);
      }
    }
    uint4* row = reinterpret_cast<uint4*>(stage + lane * 128);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float* t = v + kChunk / 8 * j;
      if constexpr (kEpi == ENC_FP8_OUT_BF16)
        row[j ^ (lane & 7)] = make_uint4(pack_bf16x2(t[0], t[1]), pack_bf16x2(t[2], t[3]), pack_bf16x2(t[4], t[5]),
                                         pack_bf16x2(t[6], t[7]));
      else
        row[j ^ (lane & 7)] = make_uint4(__float_as_uint(t[0]), __float_as_uint(t[1]), __float_as_uint(t[2]),
                                         __float_as_uint(t[3]));
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if constexpr (kEpi == ENC_FP8_OUT_RESID) tma_reduce_add_2d(map_c, stage, n0 + c, r0);
      else tma_store_2d(map_c, stage, n0 + c, r0);
      bulk_commit();
    }
  }
}

template <int kEpi, bool kGelu>
__global__ void __launch_bounds__(kThreads, 1)
gemm_fp8_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_w,
                const __grid_constant__ CUtensorMap map_c, const GemmFp8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sW = sA + kStages * kOperandBytes;
  uint8_t* stage_c = sW + kStages * kOperandBytes;                            // 4 KB per epilogue warp
  uint8_t* sS = stage_c + kEpiWarps * 4096;                                   // scale slots
  float* sB = reinterpret_cast<float*>(sS + kScaleSlots * kScaleSlotBytes);   // bias, 128 columns per epilogue warp
  uint32_t* sX = reinterpret_cast<uint32_t*>(sB + kEpiWarps * 128);           // amax of half blocks, [2][2][128]
  uint64_t* full = reinterpret_cast<uint64_t*>(sX + 512);                     // used in the first CTA
  uint64_t* empty = full + kStages;
  uint64_t* sfull = empty + kStages;        // [4] scales of both CTAs written; used in the first CTA
  uint64_t* sempty = sfull + kScaleSlots;   // [4] MMAs that read the slot are done; used in the first CTA
  uint64_t* tfull = sempty + kScaleSlots;   // [2] accumulator complete
  uint64_t* tempty = tfull + 2;             // shared columns read; used in the first CTA
  uint64_t* tdone = tempty + 1;             // [2] accumulator read; used in the first CTA
  uint64_t* drain = tdone + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
  const int units = p.num_tiles + p.tail;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int s = 0; s < kScaleSlots; ++s) { mbar_init(&sfull[s], 1); mbar_init(&sempty[s], 1); }
    for (int a = 0; a < 2; ++a) { mbar_init(&tfull[a], 1); mbar_init(&tdone[a], 2 * kEpiWarps); }
    mbar_init(tempty, 2 * kEpiWarps);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) { tma_prefetch_desc(&map_a); tma_prefetch_desc(&map_w); tma_prefetch_desc(&map_c); }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before any remote arrive or transaction
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  volatile int* abort_v = abort_flag;
  grid_dependency();   // global memory from here on

  // producer warp: bit s of `armed` = ring slot s received a load, whose phase parity is bit s of armed_phase
  uint32_t armed = 0, armed_phase = 0;
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // The whole warp walks the schedule and one elected lane issues, as for the MMAs.
    const uint32_t full_leader = peer_addr(full, 0);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = cluster; ok && u < units; u += nclusters) {
      const Unit t = unit_at(p, u);
      const int m0 = t.m0 + 128 * static_cast<int>(rank);
      // boxes of 64 rows of W: two for a full unit, one for a 128-wide one. An MMA takes its first
      // N / 2 columns' rows from the first CTA and the rest from the second, so the blocks that run as
      // N = 128 have their boxes alternate between the CTAs.
      const int early = t.width == 256 ? min(kEarly, p.num_kb) : p.num_kb;
      const uint32_t bytes = 2 * kOperandBytes + static_cast<uint32_t>(t.width) * kBK;   // of both CTAs
      for (int kb = 0; kb < p.num_kb; ++kb) {
        if (!mbar_wait_warp(&empty[stage], phase ^ 1u, abort_v, kWaitLimitNs)) { ok = false; break; }
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(&full[stage], bytes);
          const uint32_t bar = full_leader + 8 * stage;
          tma_load_2d_pair(sA + stage * kOperandBytes, &map_a, bar, kb * kBK, m0);
          const int n0 = t.n0 + (kb < early ? 64 : 128) * static_cast<int>(rank);
          tma_load_2d_pair(sW + stage * kOperandBytes, &map_w, bar, kb * kBK, n0);
          if (t.width == 256)
            tma_load_2d_pair(sW + stage * kOperandBytes + kOperandBytes / 2, &map_w, bar, kb * kBK,
                             n0 + (kb < early ? 128 : 64));
        }
        __syncwarp();
        armed |= 1u << stage;
        armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok && lane == 0) { set_status(p.status, kDevTimeout); *abort_v = 1; }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    // first CTA only: the whole warp walks the schedule, one elected lane issues
    if (leader) {
      const uint64_t adesc0 = smem_desc_sw128(smem_u32(sA)), wdesc0 = smem_desc_sw128(smem_u32(sW));
      int stage = 0, slot = 0, acc = 0;
      uint32_t phase = 0, sphase = 0, tphase = 0, dphase = 0;   // sphase: of slot 0's round
      bool ok = true, issued = false;
      bool wrapped = false;   // groups before the third have no earlier user of their TMEM columns
      // The operands of `stage` have arrived; for the first block of four also: the scales are in
      // shared memory, and the group two before, which used the same TMEM columns, is done (its
      // slot's round is the last one where slot < 2). One lane waits for each.
      auto wait_operands = [&](bool first) {
        uint64_t* bar = &full[stage];
        uint32_t parity = phase;
        if (first && lane == 1) {
          bar = &sfull[slot];
          parity = sphase;
        }
        if (first && lane == 2 && (wrapped || slot >= kScaleTmemSlots)) {
          bar = &sempty[(slot + kScaleSlots - kScaleTmemSlots) & (kScaleSlots - 1)];
          parity = sphase ^ (slot < kScaleTmemSlots ? 1u : 0u);
        }
        if (!first) return mbar_wait_warp(bar, parity, abort_v, kWaitLimitNs);
        const bool seen = __all_sync(0xffffffffu, mbar_wait<true>(bar, parity, abort_v, kWaitLimitNs));
        __syncwarp();   // what lane 1 has acquired is the issuing lane's as well
        return seen;
      };
      auto copy_scales = [&](uint32_t sfa) {
        const uint64_t sdesc = smem_desc_scales(smem_u32(sS + slot * kScaleSlotBytes));
#pragma unroll
        for (int c = 0; c < 3; ++c) tmem_cp_scales_pair(sfa + 4 * c, sdesc + c * (512 >> 4));
      };
      auto mmas = [&](uint32_t d, uint64_t ad, uint64_t wd, uint32_t idesc, uint32_t sfa, uint32_t sfb, int kb) {
#pragma unroll
        for (int k = 0; k < kBK / 32; ++k)   // +32 bytes along K inside the swizzled row
          umma_mxf8_pair(d, ad + static_cast<uint64_t>(2 * k), wd + static_cast<uint64_t>(2 * k),
                         idesc | idesc_scale_id(kb & 3), sfa, sfb, (kb | k) != 0 ? 1u : 0u);
      };
      for (int u = cluster; ok && u < units; u += nclusters) {
        const bool full_width = unit_at(p, u).width == 256;
        const int early = full_width ? min(kEarly, p.num_kb) : 0;
        // the tile two before, which used this accumulator, has been read
        if (!mbar_wait_warp(&tdone[acc], dphase ^ 1u, abort_v, kWaitLimitNs)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (acc ? kAcc1 : 0u);
        uint32_t sfa = tmem_base + kScaleCol + (slot & (kScaleTmemSlots - 1)) * kScaleSlotCols;
        // early blocks: the half without shared columns (the first one of the first accumulator)
        const int stage0 = stage;
        const uint32_t half0 = static_cast<uint32_t>(acc), half1 = 1u - half0;
        constexpr uint32_t kHalfRows = kOperandBytes >> 5;   // 64 rows, in the descriptor's units
        for (int kb = 0; kb < early; ++kb) {
          if (!wait_operands(kb == 0)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
            if (kb == 0) copy_scales(sfa);
            mmas(d_tmem + 128 * half0, adesc0 + static_cast<uint64_t>(stage) * (kOperandBytes >> 4),
                 wdesc0 + static_cast<uint64_t>(stage) * (kOperandBytes >> 4) + half0 * kHalfRows, idesc_mxf8(256, 128),
                 sfa, sfa + 4 + 4 * half0, kb);
          }
          __syncwarp();
          issued = true;
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        // the columns that the tile before shares with this one have been read
        if (!mbar_wait_warp(tempty, tphase ^ 1u, abort_v, kWaitLimitNs)) { ok = false; break; }
        tphase ^= 1u;
        tc_fence_after();
        if (early > 0) {   // their other half
          const bool last = early == p.num_kb;
          if (elect_one()) {
            int st = stage0;
            for (int e = 0; e < early; ++e) {
              mmas(d_tmem + 128 * half1, adesc0 + static_cast<uint64_t>(st) * (kOperandBytes >> 4),
                   wdesc0 + static_cast<uint64_t>(st) * (kOperandBytes >> 4) + half1 * kHalfRows, idesc_mxf8(256, 128),
                   sfa, sfa + 4 + 4 * half1, e);
              umma_commit_pair(&empty[st], 0x3);
              if (++st == kStages) st = 0;
            }
            if (last) umma_commit_pair(&sempty[slot], 0x1);
          }
          __syncwarp();
          if (last && ++slot == kScaleSlots) { slot = 0; sphase ^= 1u; wrapped = true; }
        }
        const uint32_t idesc = full_width ? idesc_mxf8(256, 256) : idesc_mxf8(256, 128);
        bool ready = false;     // the stage's operands, seen during the block before
        for (int kb = early; kb < p.num_kb; ++kb) {
          const uint32_t id = kb & 3;
          if ((id == 0 || !ready) && !wait_operands(id == 0)) { ok = false; break; }
          // the next stage's barrier is looked at here, so that its answer is there when it is needed
          const int next = stage + 1 == kStages ? 0 : stage + 1;
          ready = mbar_peek(&full[next], phase ^ (next == 0 ? 1u : 0u));
          tc_fence_after();
          sfa = tmem_base + kScaleCol + (slot & (kScaleTmemSlots - 1)) * kScaleSlotCols;
          const bool last = id == 3 || kb + 1 == p.num_kb;
          if (elect_one()) {
            if (id == 0) copy_scales(sfa);
            mmas(d_tmem, adesc0 + static_cast<uint64_t>(stage) * (kOperandBytes >> 4),
                 wdesc0 + static_cast<uint64_t>(stage) * (kOperandBytes >> 4), idesc, sfa, sfa + 4, kb);
            umma_commit_pair(&empty[stage], 0x3);
            if (last) umma_commit_pair(&sempty[slot], 0x1);
          }
          ready = __all_sync(0xffffffffu, ready);
          issued = true;
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
          if (last && ++slot == kScaleSlots) { slot = 0; sphase ^= 1u; wrapped = true; }
        }
        if (!ok) break;
        if (elect_one()) umma_commit_pair(&tfull[acc], 0x3);
        __syncwarp();
        acc ^= 1;
        if (acc == 0) dphase ^= 1u;
      }
      if (!ok && lane == 0) { set_status(p.status, kDevTimeout); *abort_v = 1; }
      if (issued) {   // every MMA done before the pair's TMEM and shared memory go away
        if (elect_one()) umma_commit_pair(drain, 0x1);
        __syncwarp();
        mbar_wait_warp(drain, 0, nullptr, kWaitLimitNs);
      }
    }
  } else if (warp < kEpiWarp0) {
    // -------------------------------------------------------------- scales
    // First CTA only: both CTAs' 128 rows of A, all the unit's rows of W for each. Two warps take
    // turns with the groups of four blocks.
    if (leader) {
      bool ok = true;
      const int groups = (p.num_kb + 3) / 4;
      const uint32_t peer = peer_addr(sS, 1) + lane * 16;
      int u = cluster, g = warp - 2;
      for (uint32_t i = warp - 2;; i += 2, g += 2) {   // the i-th group of this pair's schedule
        while (g >= groups && u < units) { g -= groups; u += nclusters; }
        if (u >= units) break;
        const Unit t = unit_at(p, u);
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 8; ++c) w[c] = scale_word(p.a_scales, p.k_pitch, t.m0 + 32 * c + lane, p.M, g);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          w[8 + c] = c * 32 < t.width ? scale_word(p.w_scales, p.k_pitch, t.n0 + 32 * c + lane, p.N, g) : kUnitScale;
        const uint32_t slot = i & (kScaleSlots - 1), sphase = (i / kScaleSlots) & 1u;
        if (!mbar_wait_warp(&sempty[slot], sphase ^ 1u, abort_v, kWaitLimitNs)) { ok = false; break; }
        uint4* dst = reinterpret_cast<uint4*>(sS + slot * kScaleSlotBytes) + lane;
        const uint32_t far = peer + slot * kScaleSlotBytes;
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        st_cluster_v4(far, make_uint4(w[4], w[5], w[6], w[7]));
#pragma unroll
        for (int c = 1; c < 3; ++c) {
          const uint4 v = make_uint4(w[4 * c + 4], w[4 * c + 5], w[4 * c + 6], w[4 * c + 7]);
          dst[c * 32] = v;
          st_cluster_v4(far + c * 512, v);
        }
        // tcgen05.cp reads them through the async proxy, in both CTAs. The arrival releases every
        // lane's stores (the warp has met) at cluster scope.
        asm volatile("fence.proxy.async;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive_release_cluster(&sfull[slot]);
      }
      if (!ok && lane == 0) { set_status(p.status, kDevTimeout); *abort_v = 1; }
    }
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;                 // TMEM lanes this warp may read
    const int half = (warp - kEpiWarp0) >> 2;     // which half of the unit's columns
    uint8_t* stage = stage_c + (warp - kEpiWarp0) * 4096;
    float* bias = sB + (warp - kEpiWarp0) * 128;
    const uint32_t tempty_leader = peer_addr(tempty, 0), tdone_leader = peer_addr(tdone, 0);
    int acc = 0;
    uint32_t tphase = 0;
    for (int u = cluster; u < units; u += nclusters) {
      const Unit t = unit_at(p, u);
      const int r0 = t.m0 + 128 * static_cast<int>(rank) + quarter * 32;
      const int per = t.width / 2, c0 = half * per, n0 = t.n0 + c0;
      float4 b4 = make_float4(0.f, 0.f, 0.f, 0.f);   // N is a multiple of 16
      if (p.bias && 4 * lane < per && n0 + 4 * lane < p.N)
        b4 = __ldg(reinterpret_cast<const float4*>(p.bias + n0) + lane);
      reinterpret_cast<float4*>(bias)[lane] = b4;    // the previous unit's reads ended with a __syncwarp
      if (!mbar_wait(&tfull[acc], tphase, abort_v, kWaitLimitNs)) {
        set_status(p.status, kDevTimeout);
        *abort_v = 1;
        // The two warps of a narrow e4m3 unit meet at a barrier that nothing bounds: there a warp that
        // gave up goes on (its output is void, and with the abort flag up its waits are short), so that
        // the other one is not left waiting.
        if constexpr (kEpi != ENC_FP8_OUT_FP8) break;
      }
      __syncwarp();
      tc_fence_after();
      bool released = false;
      auto release = [&]() {
        if (released) return;
        released = true;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader);
      };
      bool finished = false;
      auto done = [&]() {
        if (finished) return;
        finished = true;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(tdone_leader + 8 * acc);
      };
      // the first accumulator's last 32 columns are the second one's first
      const bool shares = acc ? c0 == 0 : c0 + per == 256;
      if (!shares) release();
      // of a narrow e4m3 unit both halves take part where its block of 128 columns has any
      const int first = kEpi == ENC_FP8_OUT_FP8 ? n0 & ~127 : n0;
      if (first < p.N && r0 < p.M) {
        const uint32_t taddr =
            tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + (acc ? kAcc1 : 0u) + static_cast<uint32_t>(c0);
        if constexpr (kEpi == ENC_FP8_OUT_FP8) {
          const Halves halves{sX + acc * 256, half, quarter * 32 + lane, 1 + quarter};
          if (t.width == 256)
            epilogue_e4m3<128, kGelu>(p, &map_c, r0, first, taddr, stage, bias, halves, lane, release, done);
          else   // one staging tile for both halves
            epilogue_e4m3<64, kGelu>(p, &map_c, r0, first, taddr, stage - half * (4 * 4096), bias, halves, lane,
                                     release, done);
        } else {
          epilogue<kEpi, kGelu>(p, &map_c, r0, n0, per, taddr, acc == 0, stage, bias, lane, release, done);
        }
      }
      release();
      done();
      acc ^= 1;
      if (acc == 0) tphase ^= 1u;
    }
    if (lane == 0) bulk_wait0();   // the bulk stores / reduces have landed
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0 && lane == 0 && leader && *abort_v) {
    // the first CTA's stage barriers count both CTAs' copies: after a failure, let
    // every copy issued into the pair's rings land before either CTA leaves
    for (int s = 0; s < kStages; ++s)
      if (armed & (1u << s)) mbar_wait(&full[s], (armed_phase >> s) & 1u, nullptr, kWaitLimitNs / 4);
  }
  cluster_sync();   // no CTA leaves while its pair may still read its memory
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols)
                 : "memory");
  }
}

template <int kEpi, bool kGelu>
cudaError_t launch_pair(const GemmFp8Maps& m, GemmFp8Params p, int sm_count, cudaStream_t stream) {
  static DeviceOnce once;
  static int max_clusters[64] = {};   // written under once's mutex, read after its acquire
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidValue;
  cudaError_t setup_error = cudaSuccess;
  const bool ready = once.run(dev, [&] {
    cudaError_t e = cudaFuncSetAttribute(gemm_fp8_kernel<kEpi, kGelu>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes);
    if (e != cudaSuccess) {
      setup_error = e;
      return false;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (sm_count / 2), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, gemm_fp8_kernel<kEpi, kGelu>, &cfg);
    if (e != cudaSuccess || n < 1) n = sm_count / 2;   // every SM pairs up
    cudaGetLastError();
    if (n < 1) {
      setup_error = cudaErrorInvalidValue;
      return false;
    }
    max_clusters[dev & 63] = n;
    return true;
  });
  if (!ready) return setup_error != cudaSuccess ? setup_error : cudaErrorInvalidValue;
  const int ncl = max_clusters[dev & 63];
  p.tiles_n = (p.N + 255) / 256;
  p.num_tiles = ((p.M + 255) / 256) * p.tiles_n;
  // a last wave that would run at most half full runs as two 128-wide halves per tile (of a
  // narrow last column tile the second half has no columns)
  const int tail = p.num_tiles % ncl;
  p.tail = 2 * tail <= ncl ? tail : 0;
  const int units = p.num_tiles + p.tail;
  const int clusters = units < ncl ? units : ncl;
  return launch_overlapped(gemm_fp8_kernel<kEpi, kGelu>, 2 * clusters, kThreads, kSmemBytes, 2, stream, m.a, m.w, m.c,
                           p);
}

}  // namespace

cudaError_t launch_gemm_fp8(const GemmFp8Maps& m, const GemmFp8Params& p, int out_kind, int sm_count,
                            cudaStream_t stream) {
  if (p.M <= 0) return cudaSuccess;
  switch (out_kind) {
    case ENC_FP8_OUT_BF16:
      return p.gelu ? launch_pair<ENC_FP8_OUT_BF16, true>(m, p, sm_count, stream)
                    : launch_pair<ENC_FP8_OUT_BF16, false>(m, p, sm_count, stream);
    case ENC_FP8_OUT_FP32:
      return p.gelu ? launch_pair<ENC_FP8_OUT_FP32, true>(m, p, sm_count, stream)
                    : launch_pair<ENC_FP8_OUT_FP32, false>(m, p, sm_count, stream);
    case ENC_FP8_OUT_FP8:
      return p.gelu ? launch_pair<ENC_FP8_OUT_FP8, true>(m, p, sm_count, stream)
                    : launch_pair<ENC_FP8_OUT_FP8, false>(m, p, sm_count, stream);
    case ENC_FP8_OUT_RESID: return launch_pair<ENC_FP8_OUT_RESID, false>(m, p, sm_count, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace enc
