// attn_scored_tiles.cuh — attn_scored and attn_tree with many query rows, on
// tcgen05: one CTA owns 128 query rows of one kv head (128 / G tokens x G heads)
// and walks its keys in steps of 64.
//
//   S = Q K_hat^T   M = 128, N = 64, K = D. K_hat = q d16 has up to 18
//                   significant bits and enters as an exact fp16 pair hi + lo,
//                   two products into one accumulator.
//   O += P' C       P' = p * norm as fp16 (a pair hi + lo up to head dim 128
//                   and for the rotated tiers), C the V centroids; M = 128,
//                   K = 64.
// Four roles overlap:
//   warps 0-7   softmax: two threads per row, 32 columns of S each, from TMEM;
//               cap, bias and mask in registers, P' to shared memory; the
//               running maximum moves only when it grows by 2^2 or more (O in
//               TMEM is rescaled then; P' stays below 4 norms, fp16 for any
//               norm up to a quarter of its range)
//   warps 8-15  widening: codes from global memory to fp16 operands in a ring
//               of shared-memory slots, each 128 dims of the step's K (hi, then
//               lo) or V. Two teams of four warps fill different slots at once
//               (even and odd chunks; up to head dim 128 one K and one V), since
//               a slot's time is mostly latency: the wait for the slot, the
//               table lookups, the proxy fence. Each fetches the codes of its
//               next chunk as it consumes the current one's.
//   warp 16     issues the MMAs as slots fill; a slot is free again when its
//               MMAs have completed
// S is double-buffered, so that S of the next step runs under the softmax of
// this one. At D = 512 the 512 TMEM columns hold the two S (128) and 384 output
// dims; the last 128 dims of P' C go through the S columns that the softmax has
// just read, 64 at a time, and are summed in the softmax threads' registers.
// The 128-byte-swizzle K-major layout holds every operand.
#pragma once

#include "decode_common.cuh"
#include "scored.cuh"

namespace ckv {

namespace {

template <int D, int B, int ROT>
struct CTiles {
  static constexpr int M = 128, NKV = 64;
  static constexpr int NB = D / 32;
  static constexpr int NGRP = ROT ? D / kRotGroup : 1;
  static constexpr int REC = record_bytes(D, B, NGRP);
  static constexpr int CW = D < 128 ? D : 128;      // dims per slot
  static constexpr int NCH = D / CW;                // slots per step of each operand
  static constexpr int OT = D < 384 ? D : 384;      // output dims in TMEM
  static constexpr int OR = D - OT;                 // output dims in registers
  static constexpr int NS = 2;                      // S buffers
  static constexpr int OCOL = 64 * NS;              // first O column
  static_assert(OR == 0 || OR == CW, "the tail is one slot of V");
  static constexpr bool PSPLIT = ROT || D <= 128;
  static constexpr int LUT = B == 3 ? 64 : 16;
  static constexpr int SLOT = NKV * CW * 2;
  static constexpr int P_BYTES = M * NKV * 2;
  static constexpr int Q_OFF = 0;
  static constexpr int P_OFF = M * D * 2;
  static constexpr int RING_OFF = P_OFF + (PSPLIT ? 2 : 1) * P_BYTES;
  static constexpr int TAIL = LUT * 128 + 8 * NKV * 4 + 4 * M * 4 + M * static_cast<int>(sizeof(RowInfo));
  static constexpr int BUDGET = 227 * 1024 - 1024 - 1024;  // alignment, static shared memory
  static constexpr int NSLOT_FIT = (BUDGET - RING_OFF - TAIL) / SLOT;
  static constexpr int NSLOT = NSLOT_FIT > 8 ? 8 : NSLOT_FIT;
  static_assert(NSLOT >= 3, "a K chunk takes two slots");
  static constexpr int LUT_OFF = RING_OFF + NSLOT * SLOT;
  static constexpr int NORM_OFF = LUT_OFF + LUT * 128;
  static constexpr int MAX_OFF = NORM_OFF + 8 * NKV * 4;  // norms [4][2][NKV]; [2][2][M]: the halves' row maxima, later sums
  static constexpr int ROW_OFF = MAX_OFF + 4 * M * 4;
  static constexpr int BYTES = ROW_OFF + M * static_cast<int>(sizeof(RowInfo));
  // At least half the SM's shared memory: one CTA, and its 512 TMEM columns, per SM.
  static constexpr int SMEM = (BYTES + 1024 > 120 * 1024 ? BYTES + 1024 : 120 * 1024);
  static constexpr int SOFT = 256, WIDEN = 256;     // threads of the softmax and widening roles
  static constexpr int TEAM = WIDEN / 2;
  static constexpr int THREADS = SOFT + WIDEN + 128;  // the MMA warp, in a warpgroup of its own
  // Registers per thread of the roles: 5 warpgroups are launched with 96 each.
  static constexpr int REG_SOFT = 136, REG_WIDEN = 88, REG_MMA = 32;
  static_assert(2 * REG_SOFT + 2 * REG_WIDEN + REG_MMA <= 5 * 96, "the roles share the launch's registers");
  // Output staging of the epilogue: RP rows at a time, padded by 16 bytes.
  static constexpr int STRIDE = D + 4;
  static constexpr int RP = 131 * STRIDE * 4 <= LUT_OFF ? 128 : 64 + 3 <= LUT_OFF / (STRIDE * 4) ? 64 : 32;
  static_assert((RP + 3) * STRIDE * 4 <= LUT_OFF, "staging (and the last rows' neighbours) inside the operands' memory");
};

}  // namespace

template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// umma_f16 on the low words of two 128-byte-swizzle descriptors (their high
// words are the same constant: row-group stride, version, layout).
__device__ __forceinline__ uint32_t umma_lo(uint32_t smem_addr) { return ((smem_addr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ void umma_f16_lo(uint32_t tmem_d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                            bool accumulate) {
  constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate ? 1u : 0u), "n"(kHi));
}

template <int D, int B, int ROT>
__global__ void __launch_bounds__(640, 1) attn_scored_tiles_kernel(ScoredArgs a) {
  using C = CTiles<D, B, ROT>;
  constexpr int M = C::M, NKV = C::NKV, CW = C::CW, NCH = C::NCH, NS = C::NS, NSLOT = C::NSLOT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ __align__(8) uint64_t b_full[8], b_free[8], b_sfull[2], b_sfree[2], b_pfull, b_pvdone, b_tail,
      b_tread;
  __shared__ int s_abort, s_red[4][4];
  __shared__ int8_t s_depth[64];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* const sQ = smem + C::Q_OFF;
  uint8_t* const sP = smem + C::P_OFF;
  uint8_t* const ring = smem + C::RING_OFF;
  uint32_t* const sLut = reinterpret_cast<uint32_t*>(smem + C::LUT_OFF);
  float* const sNorm = reinterpret_cast<float*>(smem + C::NORM_OFF);
  float* const sMax = reinterpret_cast<float*>(smem + C::MAX_OFF);
  RowInfo* const sRow = reinterpret_cast<RowInfo*>(smem + C::ROW_OFF);

  const int G = a.n_q_heads / a.n_kv_heads;
  const int QT = M / G;  // query tokens per tile (rows QT G .. 127 are padding)
  const int n_qt = (a.n_q + QT - 1) / QT;
  const int split = blockIdx.x % a.n_split;
  const int tile = blockIdx.x / a.n_split;
  const int qt = n_qt - 1 - tile % n_qt, bh = tile / n_qt;  // the later tokens of a prompt see more keys: first
  const int b = bh / a.n_kv_heads, kvh = bh % a.n_kv_heads;
  const int q0 = qt * QT;
  const int rows = min(QT, a.n_q - q0) * G;  // real rows of the tile
  const int act = (rows + 31) / 32;          // 32-row groups with a real row: the others' softmax warps only store

  if (warp == 0) tmem_alloc(&s_tmem, 512);
  if (tid == 32) {
    for (int s = 0; s < NSLOT; ++s) {
      mbar_init(&b_full[s], C::TEAM / 32);
      mbar_init(&b_free[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&b_sfull[s], 1);
      mbar_init(&b_sfree[s], 2 * act);
    }
    mbar_init(&b_pfull, 2 * act);
    mbar_init(&b_pvdone, 1);
    mbar_init(&b_tail, 1);
    mbar_init(&b_tread, 2 * act);
    s_abort = 0;
    fence_barrier_init();
  }
  griddep_wait();
  griddep_launch_dependents();  // the merge waits for this grid's end before it reads

  // ---- rows, their common span [glo, ghi), and the part [flo, fhi) that every row sees ----
  // Warps 0-3 form the rows while the others load Q and fill the value table.
  RowLoads in{0.0f, 0, 0, 0ull};
  if (tid < rows) in = scored_row_loads(a, b, kvh, q0 * G + tid);
  int seqlen, n;
  scored_lengths(a, b, tid == 0, seqlen, n);
  const int base = seqlen - n;
  const bool tree = a.tree != nullptr;
  if (tid < M) {
    RowInfo row{0, 0, 0, 0.0f, 0ull};
    if (tid < rows) row = scored_row(a, b, q0 * G + tid, in, seqlen, n);
    sRow[tid] = row;
    const bool some = row.lo < row.hi;
    const int lo0 = __reduce_min_sync(0xffffffffu, some ? row.lo : 0x7fffffff);
    const int hi1 = __reduce_max_sync(0xffffffffu, some ? row.hi : 0);
    const int lo1 = __reduce_max_sync(0xffffffffu, some ? row.lo : 0);
    const int hi0 = __reduce_min_sync(0xffffffffu, some ? (tree ? min(base, row.hi) : row.hi) : 0x7fffffff);
    if (lane == 0) s_red[warp][0] = lo0, s_red[warp][1] = hi1, s_red[warp][2] = lo1, s_red[warp][3] = hi0;
  } else {
    if (tid < M + 64) scored_depths(a, b, n, tid - M, s_depth);
    // Q to shared memory by asynchronous copies, all of a thread's in flight at
    // once. The splits of a tile load the same rows together: each starts at its
    // own place.
    constexpr int QTHR = C::THREADS - M, PIECES = M * (D / 8);
    const int turn0 = static_cast<int>(blockIdx.x * 37u % 64u) * (PIECES / 64);
    auto q_piece = [&](int p, int& r, int& k0) {
      const int piece = (p + turn0) % PIECES;
      r = piece / (D / 8);
      k0 = (piece % (D / 8)) * 8;
      return smem_u32(sQ) + sw128_offset(r, k0, M);
    };
#pragma unroll 4
    for (int p = tid - M; p < PIECES; p += QTHR) {
      int r, k0;
      const uint32_t dst = q_piece(p, r, k0);
      if (r < rows) {
        const __half* src = a.q + (((int64_t)b * a.n_q + q0 + r / G) * a.n_q_heads + kvh * G + r % G) * D + k0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
      } else {
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0u) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    constexpr float inv = 1.0f / centroid_scale(B);
#pragma unroll 1
    for (int e = tid - M; e < C::LUT * 32; e += QTHR) {
      const int f = e >> 5;
      const int klo = (B == 4) ? f : (f & ((1 << B) - 1));
      const int khi = (B == 4) ? f : (f >> B);
      sLut[e] = pack_half2(tbq_centroid<B>(klo) * inv, tbq_centroid<B>(khi) * inv);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (a.q_bf16) {  // to fp16 in place, each thread its own copies (exact within fp16's range)
#pragma unroll 4
      for (int p = tid - M; p < PIECES; p += QTHR) {
        int r, k0;
        const uint32_t dst = q_piece(p, r, k0);
        const uint4 v = lds128(dst);
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[e]);
          w[e] = pack_half2(__low2float(x), __high2float(x));
        }
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                     : "memory");
      }
    }
  }
  // P' of the row groups without a real row stays zero.
  for (int e = act * 32 * 8 + tid; e < M * 8; e += C::THREADS) {
    reinterpret_cast<uint4*>(sP)[e] = make_uint4(0, 0, 0, 0);
    if constexpr (C::PSPLIT) reinterpret_cast<uint4*>(sP + C::P_BYTES)[e] = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  int glo = 0x7fffffff, ghi = 0, flo = 0, fhi = 0x7fffffff;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    glo = min(glo, s_red[w][0]);
    ghi = max(ghi, s_red[w][1]);
    flo = max(flo, s_red[w][2]);
    fhi = min(fhi, s_red[w][3]);
  }
  const int lo_s = ghi > glo ? glo / NKV : 0, hi_s = ghi > glo ? (ghi + NKV - 1) / NKV : 0;
  const int s0 = lo_s + static_cast<int>((int64_t)split * (hi_s - lo_s) / a.n_split);
  const int n_steps = lo_s + static_cast<int>((int64_t)(split + 1) * (hi_s - lo_s) / a.n_split) - s0;
  const int64_t n_rec = a.capacity / kTile;
  const uint8_t* const stream = a.cache + (int64_t)(b * a.n_kv_heads + kvh) * n_rec * C::REC;

  // A wait that runs out raises the flag; every later wait is skipped, so that all roles finish.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity & 1u)) return;
    if (!*(volatile int*)&s_abort && !mbar_wait(bar, parity & 1u)) {
      *(volatile int*)&s_abort = 1;
      raise_flag(a.flag, kFlagWaitTimeout);
    }
  };

  if (tid >= C::SOFT && tid < C::SOFT + C::WIDEN) {
    // ------------------------------------------------------------ widening --
    regs_dec<C::REG_WIDEN>();
    const int team = (tid - C::SOFT) / C::TEAM, tw = (tid - C::SOFT) % C::TEAM;
    // The slots' order: K of step 0, then for every step i K of step i + 1 (all
    // but the last) and V of step i; hi and lo of a chunk are neighbours.
    auto k_index = [&](int step, int c) { return (step == 0 ? 0 : 3 * NCH * step - NCH) + 2 * c; };
    auto v_index = [&](int step, int c) { return 3 * NCH * step + (step + 1 < n_steps ? 4 : 2) * NCH + c; };
    auto slot_wait = [&](int g) {  // a slot's first use waits for the phase before its first, which passes at once
      wait(&b_free[g % NSLOT], g / NSLOT + 1);
    };
    auto slot_done = [&](int g) {
      if (lane == 0) mbar_arrive(&b_full[g % NSLOT]);
    };
    auto step_base = [&](int step) { return stream + (int64_t)(s0 + step) * (4 * C::REC); };
    // Records of a step that lie inside the cache (4 but for its end).
    auto step_recs = [&](int step) {
      return step < n_steps ? static_cast<int>(min((int64_t)4, n_rec - (int64_t)(s0 + step) * 4)) : 0;
    };
    // K chunk c of a step: 4 records x CW / 32 blocks x 32 lanes of 16 bytes,
    // each 8 dims of tokens kpp and kpp + 8 of a record. A warp has one block
    // and the records k_rec + r KS, r < KR.
    constexpr int NBLK = CW / 32, KS = 4 / NBLK, KR = 4 / KS;
    const int kq = lane >> 3, kpp = lane & 7;
    const int k_blk = (tw >> 5) % NBLK, k_rec = (tw >> 5) / NBLK;
    const int k_src = k_rec * C::REC + (k_blk * 32 + 4 * kpp + kq) * 16;
    const int k_sc = k_rec * C::REC + k_scale_offset(D) + 2 * (kpp * C::NB + k_blk);
    const uint32_t k_dst = sw128_offset(k_rec * kTile + kpp, k_blk * 32 + 8 * kq, NKV);  // + 128 per row
    uint4 kw[KR];
    uint16_t ks[KR][2];  // the two tokens' scales, as loaded: an operation on them at the fetch would wait for them there
    auto fetch_k = [&](int step, int c) {
      const uint8_t* p = step_base(step);
      const int recs = step_recs(step);
#pragma unroll
      for (int r = 0; r < KR; ++r) {
        if (k_rec + r * KS < recs) {
          const int at = r * KS * C::REC;
          kw[r] = *reinterpret_cast<const uint4*>(p + k_src + at + c * (NBLK * 512));
          const uint8_t* sc = p + k_sc + at + c * (NBLK * 2);
          ks[r][0] = *reinterpret_cast<const uint16_t*>(sc);
          ks[r][1] = *reinterpret_cast<const uint16_t*>(sc + 16 * C::NB);
        } else {
          kw[r] = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
          ks[r][0] = ks[r][1] = 0;
        }
      }
    };
    // Widens the fetched chunk c of `step` and fetches (step_n, c_n).
    auto widen_k = [&](int step, int c, int step_n, int c_n) {
      const int g = k_index(step, c);
      uint4 w4[KR];
      uint16_t sc[KR][2];
#pragma unroll
      for (int r = 0; r < KR; ++r) w4[r] = kw[r], sc[r][0] = ks[r][0], sc[r][1] = ks[r][1];
      fetch_k(step_n, c_n);
      // Both slots at once; with three slots in all, hi is handed over first and
      // lo formed after it, so that the other team's chunk can start.
      constexpr int PASSES = NSLOT < 4 ? 2 : 1;
#pragma unroll
      for (int pass = 0; pass < PASSES; ++pass) {
        slot_wait(g + pass);
        if constexpr (PASSES == 1) slot_wait(g + 1);
        uint8_t* const s_hi = ring + (g + pass) % NSLOT * C::SLOT + k_dst;
        uint8_t* const s_lo = ring + (g + 1) % NSLOT * C::SLOT + k_dst;
#pragma unroll
        for (int r = 0; r < KR; ++r) {
          const uint32_t w[4] = {w4[r].x, w4[r].y, w4[r].z, w4[r].w};
#pragma unroll
          for (int hs = 0; hs < 2; ++hs) {
            const __half2 d2 = __half2half2(__ushort_as_half(sc[r][hs]));
            uint32_t qh[4], hi[4], lo[4];
            i8x4_to_half2x2(w[2 * hs], qh[0], qh[1]);
            i8x4_to_half2x2(w[2 * hs + 1], qh[2], qh[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2 qv = *reinterpret_cast<const __half2*>(&qh[e]);
              const __half2 h = __hmul2(qv, d2);
              const __half2 l = __hfma2(qv, d2, __hneg2(h));
              hi[e] = *reinterpret_cast<const uint32_t*>(&h);
              lo[e] = *reinterpret_cast<const uint32_t*>(&l);
            }
            const int row = (r * KS * kTile + 8 * hs) * 128;
            if (pass == 0) *reinterpret_cast<uint4*>(s_hi + row) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if (pass == 1 || PASSES == 1) *reinterpret_cast<uint4*>(s_lo + row) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_proxy_async();
        __syncwarp();
        slot_done(g + pass);
        if constexpr (PASSES == 1) slot_done(g + 1);
      }
    };
    // V chunk c of a step: units of (lane stream, 8 dims), 16 fields of 2B
    // bits in B words of the stream. Unit v = 16 part + 4 record + (stream % 4),
    // part = v_part + 8 r of the chunk.
    constexpr int SUB = D / 64;                             // 8-dim parts of a lane stream
    constexpr int VR = 16 * (CW / 8) / C::TEAM;             // units per thread and chunk
    static_assert(VR >= 1, "V units per thread");
    const int v_rec = (tw >> 2) & 3, v_t = tw & 3, v_part = tw >> 4;
    constexpr int GR = v_granule(D, B);
    uint32_t vw[VR][B], vn[VR][2];
    auto fetch_v = [&](int step, int c) {
      const uint8_t* p = step_base(step) + v_rec * C::REC;
      const bool in = v_rec < step_recs(step);
#pragma unroll
      for (int r = 0; r < VR; ++r) {
        const int part = c * (CW / 8) + v_part + 8 * r;  // dims 8 part .. 8 part + 7
        const int L = 4 * (part / SUB) + v_t, w0 = (part % SUB) * B;
#pragma unroll
        for (int w = 0; w < B; ++w) {
          const int sb = 4 * (w0 + w);
          vw[r][w] = in ? *reinterpret_cast<const uint32_t*>(p + v_code_offset(D) + (sb / GR * 32 + L) * GR + sb % GR) : 0u;
        }
        if constexpr (ROT) {  // the norms of positions 2t, 2t + 1 and 2t + 8, 2t + 9
          const uint8_t* nb = p + v_norm_offset(D, B) + 2 * (kTile * (8 * part / kRotGroup) + 2 * v_t);
          vn[r][0] = in ? *reinterpret_cast<const uint32_t*>(nb) : 0u;
          vn[r][1] = in ? *reinterpret_cast<const uint32_t*>(nb + 16) : 0u;
        }
      }
    };
    auto widen_v = [&](int step, int c, int step_n, int c_n) {
      uint32_t wv[VR][B], nv[VR][2];
#pragma unroll
      for (int r = 0; r < VR; ++r) {
#pragma unroll
        for (int e = 0; e < B; ++e) wv[r][e] = vw[r][e];
        if constexpr (ROT) nv[r][0] = vn[r][0], nv[r][1] = vn[r][1];
      }
      fetch_v(step_n, c_n);
      if constexpr (ROT) {  // norms of positions that no row sees may hold any bytes; for the rest see bad_norms
        const int pos0 = (s0 + step) * NKV;
        if (pos0 < flo || pos0 + NKV > fhi) {
          uint32_t any = 0u;
          for (int rec = 0; rec < 4; ++rec) {
            uint32_t m = 0u;
            for (int r = lane; r < M; r += 32) m |= scored_tile_bits(sRow[r], tree, base, pos0 + rec * kTile);
            m = __reduce_or_sync(0xffffffffu, m);
            if (rec == v_rec) any = m;
          }
          const uint32_t ma = any >> (2 * v_t), mb = any >> (2 * v_t + 8);
#pragma unroll
          for (int r = 0; r < VR; ++r) {
            nv[r][0] = finite_norms(nv[r][0]) & ((ma & 1u ? 0xffffu : 0u) | (ma & 2u ? 0xffff0000u : 0u));
            nv[r][1] = finite_norms(nv[r][1]) & ((mb & 1u ? 0xffffu : 0u) | (mb & 2u ? 0xffff0000u : 0u));
          }
        }
      }
      const int g = v_index(step, c);
      slot_wait(g);
      const uint32_t lut = smem_u32(sLut) + (uint32_t)(lane << 2);
      // Row 8 part + d of the slot, position 16 v_rec + 2 v_t + 8 h: 16-byte
      // unit 2 v_rec + h, swizzled by the row. A warp holds two parts, whose rows
      // share their banks: one stores h while the other stores 1 - h.
      const uint32_t flip = v_part & 1;
      const uint32_t dst = smem_u32(ring + g % NSLOT * C::SLOT) + v_part * 1024 + ((2 * v_rec + flip) << 4) + 4 * v_t;
#pragma unroll
      for (int r = 0; r < VR; ++r) {
        auto field = [&](int f) {  // dim 2 (f / 4) + (f & 1), positions + 8 (f >> 1 & 1)
          uint32_t val;
          if constexpr (B == 3) {
            const int bit = 6 * f, wi = bit >> 5, sh = bit & 31;
            uint32_t y = wv[r][wi] >> sh;
            if (sh > 26 && wi + 1 < B) y |= wv[r][wi + 1 < B ? wi + 1 : wi] << (32 - sh);
            val = lds32(lut + ((y & 63u) << 7));
          } else if constexpr (B == 2) {
            val = lds32(lut + (((wv[r][f >> 3] >> (4 * (f & 7))) & 15u) << 7));
          } else {
            const uint32_t y = (wv[r][f >> 2] >> (8 * (f & 3))) & 255u;
            val = __byte_perm(lds32(lut + ((y & 15u) << 7)), lds32(lut + ((y >> 4) << 7)), 0x7610);
          }
          if constexpr (ROT) val = hmul2_u32(val, nv[r][f >> 1 & 1]);
          return val;
        };
        // Eight lookups in flight, then their stores.
#pragma unroll
        for (int f0 = 0; f0 < 16; f0 += 8) {
          uint32_t val[8];
#pragma unroll
          for (int f = 0; f < 8; ++f) val[f] = field(f0 + f);
#pragma unroll
          for (int f = 0; f < 8; ++f) {
            const int d = 2 * ((f0 + f) >> 2) + (f & 1), h = f >> 1 & 1;
            asm volatile("st.shared.u32 [%0], %1;" ::"r"((dst ^ (uint32_t)((d ^ h) << 4)) + 128 * d + 8192 * r),
                         "r"(flip ? val[f ^ 2] : val[f])
                         : "memory");
          }
        }
      }
      fence_proxy_async();
      __syncwarp();
      slot_done(g);
    };
    if constexpr (NCH == 1) {
      if (team == 0) {
        fetch_k(0, 0);
        for (int i = 0; i < n_steps; ++i) widen_k(i, 0, i + 1, 0);
      } else {
        fetch_v(0, 0);
        for (int i = 0; i < n_steps; ++i) widen_v(i, 0, i + 1, 0);
      }
    } else {
      constexpr int PER = NCH / 2;  // chunks of a step per team: team, team + 2, ...
      fetch_k(0, team);
      fetch_v(0, team);
      auto all_k = [&](int step) {
#pragma unroll 1
        for (int e = 0; e < PER; ++e)
          widen_k(step, team + 2 * e, e + 1 < PER ? step : step + 1, e + 1 < PER ? team + 2 * e + 2 : team);
      };
      if (n_steps > 0) all_k(0);
      for (int i = 0; i < n_steps; ++i) {
        if (i + 1 < n_steps) all_k(i + 1);
#pragma unroll 1
        for (int e = 0; e < PER; ++e)
          widen_v(i, team + 2 * e, e + 1 < PER ? i : i + 1, e + 1 < PER ? team + 2 * e + 2 : team);
      }
    }
    return;
  }

  if (tid >= C::SOFT + C::WIDEN) {
    // ----------------------------------------------------------------- MMA --
    regs_dec<C::REG_MMA>();
    if (warp > (C::SOFT + C::WIDEN) / 32) return;
    // The whole warp walks the schedule and one lane issues, so that the
    // operand descriptors stay in uniform registers: their low words advance
    // by constants from the operands' bases.
    const uint32_t q_lo = umma_lo(smem_u32(sQ)), p_lo = umma_lo(smem_u32(sP)), r_lo = umma_lo(smem_u32(ring));
    constexpr uint32_t kS = umma_idesc_f16_f32(M, NKV);
    int slot = 0;
    uint32_t turn = 0;
    auto slot_next = [&]() {
      if (elect_one()) umma_commit(&b_free[slot]);
      if (++slot == NSLOT) slot = 0, turn ^= 1u;
    };
    // (Rolled over the chunks: code that runs once per tile is paid for by the
    // instruction fetch, and the three roles' loops share the cache.)
    auto s_step = [&](int i) {
      const int buf = i % NS;
      if (i >= NS) wait(&b_sfree[buf], i / NS - 1);
#pragma unroll 1
      for (int c = 0; c < 2 * NCH; ++c) {  // chunk c / 2, hi then lo
        wait(&b_full[slot], turn);
        tc_fence_after();
        const uint32_t s_lo = r_lo + slot * (C::SLOT >> 4), a_lo = q_lo + (c >> 1) * ((CW / 64) * (M * 128) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < CW / 16; ++ks)
            umma_f16_lo(tmem + 64 * buf, a_lo + (((ks >> 2) * (M * 128) + (ks & 3) * 32) >> 4),
                        s_lo + (((ks >> 2) * (NKV * 128) + (ks & 3) * 32) >> 4), kS, c > 0 || ks > 0);
        }
        slot_next();
      }
      if (elect_one()) umma_commit(&b_sfull[buf]);
    };
    // O columns [col, col + N) += P' C over the step's 64 tokens, C rows from descriptor `dims`.
    auto pv = [&](uint32_t col, uint32_t dims, uint32_t idesc, bool keep) {
#pragma unroll
      for (int ks = 0; ks < NKV / 16; ++ks) {
        umma_f16_lo(tmem + col, p_lo + 2 * ks, dims + 2 * ks, idesc, keep || ks > 0);
        if constexpr (C::PSPLIT)
          umma_f16_lo(tmem + col, p_lo + (C::P_BYTES >> 4) + 2 * ks, dims + 2 * ks, idesc, true);
      }
    };
    auto pv_step = [&](int i) {
      wait(&b_pfull, i);
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        wait(&b_full[slot], turn);
        tc_fence_after();
        const uint32_t s_lo = r_lo + slot * (C::SLOT >> 4);
        if (C::OR > 0 && k == NCH - 1) {  // the tail: its first half, and once that has been read its second
          if (elect_one()) {
            pv(64 * (i % NS), s_lo, umma_idesc_f16_f32(M, 64), false);
            umma_commit(&b_tail);
          }
          wait(&b_tread, i);
          tc_fence_after();
          if (elect_one()) {
            pv(64 * (i % NS), s_lo + (64 * 128 >> 4), umma_idesc_f16_f32(M, 64), false);
            umma_commit(&b_tail);
          }
        } else if (elect_one()) {
          pv(C::OCOL + k * CW, s_lo, umma_idesc_f16_f32(M, CW), i > 0);
        }
        slot_next();
      }
      if (elect_one()) umma_commit(&b_pvdone);
    };
    if (n_steps > 0) s_step(0);
    for (int i = 0; i < n_steps; ++i) {
      if (i + 1 < n_steps) s_step(i + 1);
      pv_step(i);
    }
    __syncwarp();
    return;
  }

  // --------------------------------------------------------------- softmax --
  regs_inc<C::REG_SOFT>();
  // Softmax state: row tid % 128, columns [32 half, 32 half + 32) of every step.
  float m_used = -INFINITY, l_sum = 0.0f;
  constexpr int ORH = C::OR / 2;  // tail dims per thread: 64 part + 32 half + j at otail[32 part + j]
  float otail[C::OR > 0 ? ORH : 1];
  const int half = warp >> 2, rowi = tid & (M - 1);
  const uint32_t row_tmem = tmem + ((uint32_t)(warp & 3) * 32u << 16);

  if ((warp & 3) < act) {
    const RowInfo row = sRow[rowi];
#pragma unroll
    for (int i = 0; i < (C::OR > 0 ? ORH : 1); ++i) otail[i] = 0.0f;
    const int nk = 32 * half + lane;  // the key whose norm this thread fetches for its pair of warps
    float* const norms = sNorm + (warp & 3) * 2 * NKV;
    const uint8_t* const nbase = stream + (int64_t)s0 * (4 * C::REC) + nk / kTile * C::REC + v_norm_offset(D, B) + 2 * (nk % kTile);
    const int nkeys = seqlen - s0 * NKV - nk;  // step i has this key where 64 i < nkeys
    // As loaded: an operation on the value here would wait for it here.
    auto load_norm = [&](int step) -> uint16_t {
      return (!ROT && step < n_steps && step * NKV < nkeys)
                 ? *reinterpret_cast<const uint16_t*>(nbase + (int64_t)step * (4 * C::REC))
                 : (uint16_t)0;
    };
    // The last output dims of a step's P' C: 64 part .. of them, 32 per thread.
    auto add_tail = [&](int step, int part) {
      if constexpr (C::OR > 0) {
        wait(&b_tail, part);
        tc_fence_after();
        uint32_t tv[32];
        tmem_ld32(row_tmem + 64 * (step % NS) + 32 * half, tv);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(part ? &b_sfree[step % NS] : &b_tread);
#pragma unroll
        for (int i = 0; i < 32; ++i) otail[32 * part + i] += __uint_as_float(tv[i]);
      }
    };
    constexpr int kFormPlain = 0, kFormCap = 1, kFormAny = 2;
    const int form = a.slopes || a.cap_log2 > kShortCap || (a.cap_log2 == 0.0f && a.mul <= 0.0f) ? kFormAny
                     : a.cap_log2 > 0.0f                                                         ? kFormCap
                                                                                                 : kFormPlain;
    const float zA = form == kFormAny ? 1.0f : form == kFormCap ? -2.0f * a.cap_log2 : a.mul;
    const float zC = form == kFormCap ? a.cap_log2 : 0.0f;
    uint16_t nrm = load_norm(0);
    for (int i = 0; i < n_steps; ++i) {
      const int buf = i % NS;
      if constexpr (!ROT) {
        norms[(i & 1) * NKV + nk] = __half2float(__ushort_as_half(nrm));
        nrm = load_norm(i + 1);
      }
      const int step0 = (s0 + i) * NKV;
      const bool mixed = step0 < flo || step0 + NKV > fhi;  // some row does not see the whole step
      uint32_t gn = 0u;  // ROT, mixed: not zero where a norm of key nk is not finite
      if constexpr (ROT) {
        if (mixed && i * NKV < nkeys) {
#pragma unroll
          for (int k = 0; k < C::NGRP; ++k)
            gn |= bad_norms(*reinterpret_cast<const uint16_t*>(nbase + (int64_t)i * (4 * C::REC) + 2 * kTile * k));
        }
      }
      if (i > 0) {  // at once: S of the next step waits for these columns
        add_tail(i - 1, 0);
        add_tail(i - 1, 1);
      }
      wait(&b_sfull[buf], i / NS);
      tc_fence_after();
      uint32_t sv[32];
      tmem_ld32(row_tmem + 64 * buf + 32 * half, sv);
      tmem_ld_wait();
      if constexpr (C::OR == 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_sfree[buf]);
      }
      // z of each key, with the logit = A z + C: S itself, the 1 / (1 + e^2x) of
      // a short cap, or (distance bias, long cap, negative scale) the logit. (A
      // polynomial tanh on [-1, 1], nine packed operations a pair in place of
      // the exponential and the reciprocal, took 1598 cycles a step against 1217.)
      float z[32], mx;
      const int p0 = (s0 + i) * NKV + 32 * half;
      uint32_t see = row.hi > 0 ? ~0u : 0u;
      if (mixed) see = static_cast<uint32_t>(scored_step_bits(row, tree, base, p0));
      const bool masked = __any_sync(0xffffffffu, see != ~0u);
      if (form == kFormCap) {
        const uint64_t k2 = f32x2(a.mul * 2.8853900817779268f, a.mul * 2.8853900817779268f), one = f32x2(1.0f, 1.0f);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float2 y = f32x2_get(mul_f32x2(f32x2(__uint_as_float(sv[j]), __uint_as_float(sv[j + 1])), k2));
          const float2 d = f32x2_get(add_f32x2(f32x2(fast_exp2(y.x), fast_exp2(y.y)), one));
          z[j] = fast_rcp(d.x);
          z[j + 1] = fast_rcp(d.y);
        }
      } else if (form == kFormPlain) {
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(sv[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j] = scored_logit(__uint_as_float(sv[j]), a.mul, a.cap_log2);
        if (tree && p0 + 32 > base) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            z[j] = fmaf(-row.slope, static_cast<float>(abs(row.at - scored_key_at(s_depth, tree, base, p0 + j))), z[j]);
        } else {
          const float d0 = static_cast<float>(row.at - p0);
#pragma unroll
          for (int j = 0; j < 32; ++j) z[j] = fmaf(-row.slope, fabsf(d0 - static_cast<float>(j)), z[j]);
        }
      }
      if (masked) {
        const float never = form == kFormCap ? INFINITY : -INFINITY;
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j] = (see >> j & 1u) ? z[j] : never;
      }
      if (form == kFormCap) {
        float t0 = z[0], t1 = z[1];
#pragma unroll
        for (int j = 2; j < 32; j += 4) {
          t0 = min3(t0, z[j], z[j + 1]);
          if (j + 2 < 32) t1 = min3(t1, z[j + 2], z[j + 3]);
        }
        mx = fmaf(zA, fminf(t0, t1), zC);
      } else {
        float t0 = z[0], t1 = z[1];
#pragma unroll
        for (int j = 2; j < 32; j += 4) {
          t0 = max3(t0, z[j], z[j + 1]);
          if (j + 2 < 32) t1 = max3(t1, z[j + 2], z[j + 3]);
        }
        mx = zA * fmaxf(t0, t1);
      }
      float* const ex = sMax + (i & 1) * 2 * M + rowi;
      ex[half * M] = mx;
      named_bar(1 + (warp & 3), 64);  // the row's two warps
      mx = fmaxf(mx, ex[(1 - half) * M]);
      // P' and (for a rescale) O are free once the step before has been multiplied.
      if (i > 0) wait(&b_pvdone, i - 1);
      tc_fence_after();
      const bool need = mx > m_used + 2.0f;  // also when m_used is -inf and a key is seen
      if (__any_sync(0xffffffffu, need)) {
        const float f = need ? ((m_used == -INFINITY) ? 0.0f : fast_exp2(m_used - mx)) : 1.0f;
        if (i > 0) {
#pragma unroll 1
          for (int c0 = C::OCOL + half * (C::OT / 2); c0 < C::OCOL + (half + 1) * (C::OT / 2); c0 += 32) {
            uint32_t ov[32];
            tmem_ld32(row_tmem + c0, ov);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * f);
            tmem_st32(row_tmem + c0, ov);
          }
          tmem_st_wait();
        }
#pragma unroll
        for (int k = 0; k < ORH; ++k) otail[k] *= f;
        l_sum *= f;
        if (need) m_used = mx;
      }
      const float mref = (m_used == -INFINITY) ? 0.0f : m_used;  // nothing seen yet: every x is -inf
      uint64_t ps = f32x2(0.0f, 0.0f);
      const uint64_t zA2 = f32x2(zA, zA), zC2 = f32x2(zC - mref, zC - mref);
      const float4* n4 = reinterpret_cast<const float4*>(norms + (i & 1) * NKV + 32 * half);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = 8 * c + 4 * h;
          const float2 xa = f32x2_get(fma_f32x2(zA2, f32x2(z[j], z[j + 1]), zC2));
          const float2 xb = f32x2_get(fma_f32x2(zA2, f32x2(z[j + 2], z[j + 3]), zC2));
          uint64_t ya = f32x2(fast_exp2(xa.x), fast_exp2(xa.y)), yb = f32x2(fast_exp2(xb.x), fast_exp2(xb.y));
          ps = add_f32x2(ps, add_f32x2(ya, yb));
          if constexpr (!ROT) {
            float4 nn = n4[2 * c + h];
            if (masked) {  // the norm of a key that the row does not see may hold any bytes
              nn.x = (see >> j & 1u) ? nn.x : 0.0f;
              nn.y = (see >> (j + 1) & 1u) ? nn.y : 0.0f;
              nn.z = (see >> (j + 2) & 1u) ? nn.z : 0.0f;
              nn.w = (see >> (j + 3) & 1u) ? nn.w : 0.0f;
            }
            ya = mul_f32x2(ya, f32x2(nn.x, nn.y));
            yb = mul_f32x2(yb, f32x2(nn.z, nn.w));
          }
          const float2 fa = f32x2_get(ya), fb = f32x2_get(yb);
          hi[2 * h] = pack_half2(fa.x, fa.y);
          hi[2 * h + 1] = pack_half2(fb.x, fb.y);
          if constexpr (C::PSPLIT) {
            const float2 ha = __half22float2(*reinterpret_cast<const __half2*>(&hi[2 * h]));
            const float2 hb = __half22float2(*reinterpret_cast<const __half2*>(&hi[2 * h + 1]));
            lo[2 * h] = pack_half2(fa.x - ha.x, fa.y - ha.y);
            lo[2 * h + 1] = pack_half2(fb.x - hb.x, fb.y - hb.y);
          }
        }
        const uint32_t off = sw128_offset(rowi, 32 * half + 8 * c, M);
        *reinterpret_cast<uint4*>(sP + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if constexpr (C::PSPLIT)
          *reinterpret_cast<uint4*>(sP + C::P_BYTES + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      if constexpr (ROT) {
        uint32_t bad = mixed ? __ballot_sync(0xffffffffu, gn != 0u) & see : 0u;
        while (bad) {  // NaN for the keys that this row sees and whose norm left V
          const int j = __ffs(bad) - 1;
          bad &= bad - 1u;
          *reinterpret_cast<uint16_t*>(sP + sw128_offset(rowi, 32 * half + (j & ~7), M) + 2 * (j & 7)) = 0x7fffu;
        }
      }
      const float2 p2 = f32x2_get(ps);
      l_sum += p2.x + p2.y;
      fence_proxy_async();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b_pfull);
    }
    if (n_steps > 0) {
      add_tail(n_steps - 1, 0);
      add_tail(n_steps - 1, 1);
      wait(&b_pvdone, n_steps - 1);
      tc_fence_after();
    }
    // The row's sum: both halves'.
    float* const ex = sMax + (n_steps & 1) * 2 * M + rowi;
    ex[half * M] = l_sum;
    named_bar(1 + (warp & 3), 64);  // the row's two warps
    l_sum += ex[(1 - half) * M];
  }

  // ---------------------------------------------------------------- epilogue --
  // Rows leave TMEM one per thread; they cross to one row per warp through the
  // operands' shared memory, C::RP rows at a time, there get the inverse
  // transform (one split) and go out in whole lines.
  const bool direct = a.n_split == 1;
  float* const slot = a.part + (int64_t)blockIdx.x * (M * (D + 1));
  float* const stage = reinterpret_cast<float*>(smem);
  const float inv = row_inv<true>(l_sum);
  if (tid < rows) {
    const float lse = row_lse<true>(m_used, l_sum);
    if (direct) a.lse[((int64_t)b * a.n_q + q0 + tid / G) * a.n_q_heads + kvh * G + tid % G] = lse;
    else slot[(int64_t)M * D + tid] = lse;
  }
  tc_fence_before();
  named_bar(5, C::SOFT);
  tc_fence_after();
  for (int r0 = 0; r0 < rows; r0 += C::RP) {
    if ((warp & 3) < act && (warp & 3) * 32 >= r0 && (warp & 3) * 32 < r0 + C::RP) {
      float* const dst = stage + (rowi - r0) * C::STRIDE;
#pragma unroll 1
      for (int c = half * (C::OT / 2); c < (half + 1) * (C::OT / 2); c += 32) {
        uint32_t ov[32];
        if (n_steps > 0) {
          tmem_ld32(row_tmem + C::OCOL + c, ov);
          tmem_ld_wait();
        }
#pragma unroll
        for (int k = 0; k < 32; k += 4)
          *reinterpret_cast<float4*>(dst + c + k) =
              inv != 0.0f ? make_float4(__uint_as_float(ov[k]) * inv, __uint_as_float(ov[k + 1]) * inv,
                                       __uint_as_float(ov[k + 2]) * inv, __uint_as_float(ov[k + 3]) * inv)
                         : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      if constexpr (C::OR > 0) {
#pragma unroll
        for (int k = 0; k < ORH; k += 4)
          *reinterpret_cast<float4*>(dst + C::OT + 64 * (k / 32) + 32 * half + k % 32) =
              inv != 0.0f ? make_float4(otail[k] * inv, otail[k + 1] * inv, otail[k + 2] * inv, otail[k + 3] * inv)
                         : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
    }
    named_bar(5, C::SOFT);
    // A warp takes RPW rows together: a row alone is a chain of shuffles.
    constexpr int RPW = D == 512 ? 1 : D == 256 ? 2 : 4, WARPS = C::SOFT / 32;
    for (int rw = r0 + RPW * warp; rw < min(rows, r0 + C::RP); rw += RPW * WARPS) {
      float2 v[RPW][D / 64];
#pragma unroll
      for (int k = 0; k < RPW; ++k)
#pragma unroll
        for (int e = 0; e < D / 64; ++e)
          v[k][e] = *reinterpret_cast<const float2*>(stage + (rw + k - r0) * C::STRIDE + 64 * e + 2 * lane);
      float* o[RPW];
#pragma unroll
      for (int k = 0; k < RPW; ++k) {
        const int r = rw + k;
        const int64_t orow = ((int64_t)b * a.n_q + q0 + r / G) * a.n_q_heads + kvh * G + r % G;
        float* const to = !direct                   ? slot + (int64_t)r * D
                          : a.out_type == kOutF32 ? a.out + orow * D
                                                  : reinterpret_cast<float*>(reinterpret_cast<uint16_t*>(a.out) + orow * D);
        o[k] = r < rows ? to : nullptr;
      }
      if (direct) derotate_rows<D, ROT, RPW>(v, lane, a.signs, centroid_scale(B), a.signs2);
#pragma unroll
      for (int k = 0; k < RPW; ++k)
        if (o[k])
#pragma unroll
          for (int e = 0; e < D / 64; ++e) store_out2<true>(o[k], lane + 32 * e, v[k][e], direct ? a.out_type : kOutF32);
    }
    named_bar(5, C::SOFT);
  }
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// The n_split partials of every output row, merged exactly (log-sum-exp), and
// the inverse transform: one CTA per row. The partials sit in L2: every thread
// takes one 16-byte unit of the row over a strided subset of the slots with all
// its loads (up to 20) in flight before the weights are known, so that the
// merge costs about one round trip.
constexpr int kScoredMergeThreads = 512;
template <int D, int B, int ROT>
__global__ void __launch_bounds__(kScoredMergeThreads) scored_merge_rows_kernel(ScoredArgs a) {
  constexpr int M = 128, NT = kScoredMergeThreads, UNITS = D / 4, SG = NT / UNITS, PER = 20;
  constexpr int64_t SLOT = M * (int64_t)(D + 1);
  __shared__ float s_w[kMaxSplits];
  __shared__ float s_red[NT / 32];
  __shared__ __align__(16) float4 s_acc[SG][UNITS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  const int G = a.n_q_heads / a.n_kv_heads, QT = M / G, n_qt = (a.n_q + QT - 1) / QT;
  const int64_t r = blockIdx.x;
  const int h = static_cast<int>(r % a.n_q_heads);
  const int64_t bq = r / a.n_q_heads;
  const int qi = static_cast<int>(bq % a.n_q), b = static_cast<int>(bq / a.n_q);
  const int64_t tile = ((int64_t)b * a.n_kv_heads + h / G) * n_qt + (n_qt - 1 - qi / QT);
  const int rin = (qi % QT) * G + h % G, n_split = a.n_split;
  const float* const base = a.part + tile * n_split * SLOT;
  const int u = tid % UNITS, g = tid / UNITS;
  float4 x[PER];
  auto load = [&](int s0) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int s = s0 + g + j * SG;
      if (s < n_split) x[j] = __ldcg(reinterpret_cast<const float4*>(base + s * SLOT + (int64_t)rin * D) + u);
    }
  };
  load(0);
  float m = -INFINITY;
  for (int s = tid; s < n_split; s += NT) {
    const float l = __ldcg(base + s * SLOT + (int64_t)M * D + rin);
    s_w[s] = l;
    m = fmaxf(m, l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s_red[warp] = m;
  __syncthreads();
  m = s_red[0];
#pragma unroll
  for (int w = 1; w < NT / 32; ++w) m = fmaxf(m, s_red[w]);
  for (int s = tid; s < n_split; s += NT) s_w[s] = (s_w[s] == -INFINITY) ? 0.0f : exp2f((s_w[s] - m) * 1.4426950408889634f);
  __syncthreads();
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s0 = 0; s0 < n_split; s0 += PER * SG) {
    if (s0 > 0) load(s0);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int s = s0 + g + j * SG;
      if (s < n_split) {
        const float w = s_w[s];
        acc.x = fmaf(w, x[j].x, acc.x);
        acc.y = fmaf(w, x[j].y, acc.y);
        acc.z = fmaf(w, x[j].z, acc.z);
        acc.w = fmaf(w, x[j].w, acc.w);
      }
    }
  }
  s_acc[g][u] = acc;
  __syncthreads();
  if (warp) return;
  float total = 0.0f;
  for (int s = lane; s < n_split; s += 32) total += s_w[s];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const float inv = row_inv<true>(total);
  const float* flat = reinterpret_cast<const float*>(s_acc);
  float2 v[D / 64];
#pragma unroll
  for (int e = 0; e < D / 64; ++e) {
    float2 y = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < SG; ++k) {
      const float2 z = *reinterpret_cast<const float2*>(flat + k * D + 64 * e + 2 * lane);
      y.x += z.x;
      y.y += z.y;
    }
    v[e] = make_float2(y.x * inv, y.y * inv);
  }
  float* const o = a.out_type == kOutF32 ? a.out + r * D
                                         : reinterpret_cast<float*>(reinterpret_cast<uint16_t*>(a.out) + r * D);
  derotate_store_row<D, ROT, true>(v, lane, a.signs, o, centroid_scale(B), a.signs2, a.out_type);
  if (lane == 0) a.lse[r] = total != 0.0f ? m + logf(total) : -INFINITY;
}

// The same for few splits (at most 32), where rows are many: one warp per row.
template <int D, int B, int ROT>
__global__ void __launch_bounds__(256) scored_merge_few_kernel(ScoredArgs a) {
  constexpr int M = 128, PER = 4;
  constexpr int64_t SLOT = M * (int64_t)(D + 1);
  const int lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  griddep_wait();
  if (r >= (int64_t)a.batch * a.n_q * a.n_q_heads) return;
  const int G = a.n_q_heads / a.n_kv_heads, QT = M / G, n_qt = (a.n_q + QT - 1) / QT;
  const int h = static_cast<int>(r % a.n_q_heads);
  const int64_t bq = r / a.n_q_heads;
  const int qi = static_cast<int>(bq % a.n_q), b = static_cast<int>(bq / a.n_q);
  const int64_t tile = ((int64_t)b * a.n_kv_heads + h / G) * n_qt + (n_qt - 1 - qi / QT);
  const int rin = (qi % QT) * G + h % G;
  const float* const base = a.part + tile * a.n_split * SLOT;
  const float l = lane < a.n_split ? __ldcg(base + lane * SLOT + (int64_t)M * D + rin) : -INFINITY;
  float m = l;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float w = (l == -INFINITY) ? 0.0f : exp2f((l - m) * 1.4426950408889634f);
  float total = w;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const float inv = row_inv<true>(total);
  float2 v[D / 64];
#pragma unroll
  for (int e = 0; e < D / 64; ++e) v[e] = make_float2(0.0f, 0.0f);
  for (int s0 = 0; s0 < a.n_split; s0 += PER) {
    float2 x[PER][D / 64];
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (s0 + j < a.n_split) {
        const float2* src = reinterpret_cast<const float2*>(base + (s0 + j) * SLOT + (int64_t)rin * D) + lane;
#pragma unroll
        for (int e = 0; e < D / 64; ++e) x[j][e] = __ldcg(src + 32 * e);
      }
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (s0 + j < a.n_split) {
        const float ws = __shfl_sync(0xffffffffu, w, s0 + j) * inv;
#pragma unroll
        for (int e = 0; e < D / 64; ++e) {
          v[e].x = fmaf(ws, x[j][e].x, v[e].x);
          v[e].y = fmaf(ws, x[j][e].y, v[e].y);
        }
      }
  }
  float* const o = a.out_type == kOutF32 ? a.out + r * D
                                         : reinterpret_cast<float*>(reinterpret_cast<uint16_t*>(a.out) + r * D);
  derotate_store_row<D, ROT, true>(v, lane, a.signs, o, centroid_scale(B), a.signs2, a.out_type);
  if (lane == 0) a.lse[r] = total != 0.0f ? m + logf(total) : -INFINITY;
}

template <int D, int B, int ROT>
static cudaError_t launch_scored_tiles_d(const ScoredArgs& a, cudaStream_t stream) {
  using C = CTiles<D, B, ROT>;
  static bool configured[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !configured[dev]) {
    e = cudaFuncSetAttribute(attn_scored_tiles_kernel<D, B, ROT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) configured[dev] = true;
  }
  const int QT = C::M / (a.n_q_heads / a.n_kv_heads), n_qt = (a.n_q + QT - 1) / QT;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((int64_t)a.batch * a.n_kv_heads * n_qt * a.n_split));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attn_scored_tiles_kernel<D, B, ROT>, a);
  if (e != cudaSuccess || a.n_split == 1) return e;
  const int64_t out_rows = (int64_t)a.batch * a.n_q * a.n_q_heads;
  cfg.dynamicSmemBytes = 0;
  if (a.n_split <= 32) {
    cfg.gridDim = dim3(static_cast<unsigned>((out_rows + 7) / 8));
    cfg.blockDim = dim3(256);
    return cudaLaunchKernelEx(&cfg, scored_merge_few_kernel<D, B, ROT>, a);
  }
  cfg.gridDim = dim3(static_cast<unsigned>(out_rows));
  cfg.blockDim = dim3(kScoredMergeThreads);
  return cudaLaunchKernelEx(&cfg, scored_merge_rows_kernel<D, B, ROT>, a);
}

}  // namespace ckv
