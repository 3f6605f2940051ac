// attn_scored_kernel.cuh — attn_scored and attn_tree with few query rows, on
// mma.sync: the split-K decode over the packed records with scored.cuh's masks
// and logits, one row group (8 query rows of one kv head) per CTA. Every tile
// group (a warp, or two at D = 512) streams its own records through its own
// stages, so no warp waits for another but its partner.
//
// Mathematics: the decode kernel's (S^T = K_hat Q^T and O^T += C^T P'^T, the
// codes widened in registers, one online softmax over the row's keys), with
// x = c tanh(mul S) - slope |distance| between the product and the softmax.
#pragma once

#include "attn_decode_kernel.cuh"
#include "attn_scored_tiles.cuh"
#include "scored.cuh"

namespace ckv {

namespace {

// Warps per CTA: twelve at head dim 512 (168 registers a thread; a 32768-token
// step 21.0 us against 22.0 with eight), else eight. At head dim 256 a second
// CTA per SM would spill (a windowed batch 51.8 us against 37.2).
constexpr int scored_warps(int D) { return D == 512 ? 12 : 8; }

template <int D, int B, int ROT>
struct CScored : DecodeShape<D, scored_warps(D)> {
  using Sh = DecodeShape<D, scored_warps(D)>;
  static constexpr int NGRP = ROT ? D / kRotGroup : 1;
  static constexpr int REC = record_bytes(D, B, NGRP);
  static constexpr int NSTAGE = D == 512 ? 2 : 4;  // records in flight per tile group
  static constexpr int THREADS = Sh::NCW * 32;
  // The rotated tiers round V's fragments to fp16 once more (the group norms
  // scale them), so their P' is always the fp16 pair.
  static constexpr bool PSPLIT = ROT || D <= 128;
  static constexpr int LUT = CDec<D, B, ROT>::LUT;
  static constexpr int RED_BYTES = Sh::NP * Sh::RED_FLOATS * 4;
  static constexpr int RING = (Sh::NP * NSTAGE * REC > RED_BYTES) ? Sh::NP * NSTAGE * REC : RED_BYTES;
  static constexpr int OFF_XCHG = (RING + 127) / 128 * 128;
  static constexpr int OFF_ML = OFF_XCHG + Sh::XCHG_BYTES;
  static constexpr int OFF_QB = OFF_ML + Sh::NP * 16 * 4;
  static constexpr int OFF_BAR = OFF_QB + Sh::NCW * Sh::NB_W * 4 * 2 * 4;
  static constexpr int SMEM = OFF_BAR + Sh::NP * NSTAGE * 8 + 16;
  // Up to head dim 128 the accumulators leave the registers for a second CTA on the SM.
  static constexpr int PER_SM = D <= 128 ? 2 : 1;
  static_assert(PER_SM * (SMEM + LUT * 128 + 4096) <= 227 * 1024, "shared memory");
};

// load_q_frags for bf16 queries, converted to fp16 (exact within fp16's range).
template <int NBW>
__device__ __forceinline__ void convert_q_frags(uint32_t (&qf)[NBW][4]) {
#pragma unroll
  for (int i = 0; i < NBW; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&qf[i][j]);
      qf[i][j] = pack_half2(__low2float(x), __high2float(x));
    }
}

}  // namespace

template <int D, int B, int ROT>
__global__ void __launch_bounds__(CScored<D, B, ROT>::THREADS, CScored<D, B, ROT>::PER_SM)
    attn_scored_kernel(ScoredArgs a) {
  using C = CScored<D, B, ROT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) uint32_t s_lut[C::LUT * 32];
  __shared__ RowInfo s_row[8];
  __shared__ int8_t s_depth[64];
  __shared__ int s_abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x, rg = blockIdx.y, bh = blockIdx.z;
  const int b = bh / a.n_kv_heads, kvh = bh % a.n_kv_heads;
  const int group_q = a.n_q_heads / a.n_kv_heads;
  const int R = group_q * a.n_q;

  const int group = warp / C::WT, wh = warp % C::WT;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + group * C::NSTAGE;
  float4* xbuf = reinterpret_cast<float4*>(smem + C::OFF_XCHG);
  float* mlbuf = reinterpret_cast<float*>(smem + C::OFF_ML);

  // Before the previous grid on the stream has finished: barriers and table.
  if (threadIdx.x == 0) {
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    for (int s = 0; s < C::NP * C::NSTAGE; ++s) mbar_init(&bars[s], 1);
    s_abort = 0;
    fence_barrier_init();
  }
  {
    constexpr float inv = 1.0f / centroid_scale(B);
    for (int e = threadIdx.x; e < C::LUT * 32; e += C::THREADS) {
      const int f = e >> 5;
      const int klo = (B == 4) ? f : (f & ((1 << B) - 1));
      const int khi = (B == 4) ? f : (f >> B);
      s_lut[e] = pack_half2(tbq_centroid<B>(klo) * inv, tbq_centroid<B>(khi) * inv);
    }
  }
  griddep_wait();
  griddep_launch_dependents();

  uint32_t qf[C::NB_W][4];
  {
    const int rr = rg * 8 + (lane >> 2);
    int qi = 0, h = 0;
    const bool ok = rr < R;
    if (ok) row_to_query(rr, group_q, kvh, qi, h);
    load_q_frags<C::NB_W>(qf, a.q + ((int64_t)(b * a.n_q + qi) * a.n_q_heads + h) * D, ok, wh * C::NB_W, lane & 3);
    if (a.q_bf16) convert_q_frags<C::NB_W>(qf);
  }
  RowLoads in{0.0f, 0, 0, 0ull};
  if (threadIdx.x < 8) in = scored_row_loads(a, b, kvh, rg * 8 + threadIdx.x);
  int seqlen, n;
  scored_lengths(a, b, threadIdx.x == 0, seqlen, n);
  const int base = seqlen - n;
  if (threadIdx.x < 8) s_row[threadIdx.x] = scored_row(a, b, rg * 8 + threadIdx.x, in, seqlen, n);
  if (warp >= 2 && warp < 4) scored_depths(a, b, n, threadIdx.x - 64, s_depth);
  __syncthreads();

  // The CTA's keys: the union [glo, ghi) of its rows' intervals, cut into
  // n_split runs of tiles; the tiles inside [flo, fhi) are seen whole by every
  // row that sees anything.
  int glo = 0x7fffffff, ghi = 0, flo = 0, fhi = 0x7fffffff;
  for (int r = 0; r < 8; ++r) {
    const int lo = s_row[r].lo, hi = s_row[r].hi;
    if (lo < hi) {
      glo = min(glo, lo);
      ghi = max(ghi, hi);
      flo = max(flo, lo);
      fhi = min(fhi, a.tree ? min(base, hi) : hi);
    }
  }
  const int64_t lo_t = ghi > glo ? glo / kTile : 0, hi_t = ghi > glo ? (ghi + kTile - 1) / kTile : 0;
  const int64_t tb = lo_t + (int64_t)split * (hi_t - lo_t) / a.n_split;
  const int64_t te = lo_t + (int64_t)(split + 1) * (hi_t - lo_t) / a.n_split;
  // This group's tiles: tb + group, + NP, ... below te, each one record, one
  // bulk copy and one stage of the group's own ring.
  const int n_iters = te > tb + group ? static_cast<int>((te - tb - group + C::NP - 1) / C::NP) : 0;
  const uint8_t* gbase = a.cache + (int64_t)(b * a.n_kv_heads + kvh) * (a.capacity / kTile) * C::REC;
  uint8_t* const gring = smem + group * C::NSTAGE * C::REC;
  auto issue = [&](int it) {  // one lane of the group
    const int s = it % C::NSTAGE;
    mbar_arrive_expect_tx(&full[s], C::REC);
    bulk_g2s(gring + s * C::REC, gbase + (tb + group + (int64_t)it * C::NP) * C::REC, C::REC, &full[s]);
  };
  const bool leader = wh == 0 && lane == 0;
  if (leader)
    for (int it = 0; it < n_iters && it < C::NSTAGE; ++it) issue(it);

  const int g = lane >> 2, t = lane & 3;
  float* qb_warp = reinterpret_cast<float*>(smem + C::OFF_QB) + warp * C::NB_W * 8;
  q_block_bias<C::NB_W>(qf, lane, qb_warp);
  const uint32_t qb = smem_u32(qb_warp) + t * 8;
  const RowInfo mine = s_row[lane % (8)];  // the row whose masks this lane forms
  const int at0 = s_row[2 * t].at, at1 = s_row[2 * t + 1].at;
  const float sl0 = s_row[2 * t].slope, sl1 = s_row[2 * t + 1].slope;
  const bool tree = a.tree != nullptr, biased = a.slopes != nullptr;
  float acc[C::MT_W][4];
#pragma unroll
  for (int i = 0; i < C::MT_W; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
  SoftmaxState st{-INFINITY, -INFINITY, 0.0f, 0.0f};

  const uint32_t ring = smem_u32(gring);
  const uint8_t* lut_bytes = reinterpret_cast<const uint8_t*>(s_lut);
  const uint32_t lane4 = (uint32_t)lane << 2;

  auto wait_stage = [&](int it) {
    if (!*(volatile int*)&s_abort) {
      if (!mbar_wait(&full[it % C::NSTAGE], (it / C::NSTAGE) & 1)) {
        *(volatile int*)&s_abort = 1;
        raise_flag(a.flag, kFlagWaitTimeout);
      }
    }
  };
  auto record = [&](int it) { return ring + (it % C::NSTAGE) * C::REC; };
  // S of the next tile is in flight under the softmax and P.V of this one (two
  // warps to a tile: each one's half crosses through shared memory).
  float S[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (n_iters > 0) {
    wait_stage(0);
    qk_tile<D>(record(0), wh, lane, qf, qb, S);
    if constexpr (C::WT == 2) exchange_S<2>(S, xbuf, group, wh, 0, lane);
  }
  for (int it = 0; it < n_iters; ++it) {
    const int64_t tile = tb + (int64_t)it * C::NP + group;
    const bool next = it + 1 < n_iters;
    float Sn[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (next) {
      wait_stage(it + 1);
      qk_tile<D>(record(it + 1), wh, lane, qf, qb, Sn);
      if constexpr (C::WT == 2) xchg_put<2>(Sn, xbuf, group, wh, (it + 1) & 1, lane);
    }
    {
      const uint32_t rb = record(it);
      const int64_t tpos = tile * kTile;
      // Visibility: position tpos + g is bit g of its row's word, tpos + g + 8 bit g + 8.
      uint32_t v0 = 0xffffu, v1 = 0xffffu, any = 0xffffu;
      const bool mixed = tpos < flo || tpos + kTile > fhi;
      if (mixed) {
        const uint32_t bits = scored_tile_bits(mine, tree, base, tpos);
        v0 = __shfl_sync(0xffffffffu, bits, 2 * t);
        v1 = __shfl_sync(0xffffffffu, bits, 2 * t + 1);
        any = __reduce_or_sync(0xffffffffu, bits);
      }
      const bool s0 = v0 >> g & 1u, s1 = v1 >> g & 1u, s2 = v0 >> (g + 8) & 1u, s3 = v1 >> (g + 8) & 1u;
      float x0 = scored_logit(S[0], a.mul, a.cap_log2), x1 = scored_logit(S[1], a.mul, a.cap_log2);
      float x2 = scored_logit(S[2], a.mul, a.cap_log2), x3 = scored_logit(S[3], a.mul, a.cap_log2);
      if (biased) {
        const int ka = scored_key_at(s_depth, tree, base, static_cast<int>(tpos) + g);
        const int kb = scored_key_at(s_depth, tree, base, static_cast<int>(tpos) + g + 8);
        x0 = fmaf(-sl0, static_cast<float>(abs(at0 - ka)), x0);
        x1 = fmaf(-sl1, static_cast<float>(abs(at1 - ka)), x1);
        x2 = fmaf(-sl0, static_cast<float>(abs(at0 - kb)), x2);
        x3 = fmaf(-sl1, static_cast<float>(abs(at1 - kb)), x3);
      }
      x0 = s0 ? x0 : -INFINITY;
      x1 = s1 ? x1 : -INFINITY;
      x2 = s2 ? x2 : -INFINITY;
      x3 = s3 ? x3 : -INFINITY;
      const float mn0 = fmaxf(st.m0, warp_max_over_gid(fmaxf(x0, x2)));
      const float mn1 = fmaxf(st.m1, warp_max_over_gid(fmaxf(x1, x3)));
      if (__any_sync(0xffffffffu, (mn0 > st.m0) || (mn1 > st.m1))) {
        const float a0 = (st.m0 == -INFINITY) ? 0.0f : fast_exp2(st.m0 - mn0);
        const float a1 = (st.m1 == -INFINITY) ? 0.0f : fast_exp2(st.m1 - mn1);
#pragma unroll
        for (int i = 0; i < C::MT_W; ++i) {
          acc[i][0] *= a0;
          acc[i][1] *= a1;
          acc[i][2] *= a0;
          acc[i][3] *= a1;
        }
        st.l0 *= a0;
        st.l1 *= a1;
        st.m0 = mn0;
        st.m1 = mn1;
      }
      const float p0 = s0 ? fast_exp2(x0 - st.m0) : 0.0f, p1 = s1 ? fast_exp2(x1 - st.m1) : 0.0f;
      const float p2 = s2 ? fast_exp2(x2 - st.m0) : 0.0f, p3 = s3 ? fast_exp2(x3 - st.m1) : 0.0f;
      st.l0 += p0 + p2;
      st.l1 += p1 + p3;

      // V's norms: folded into P', or (ROT) into V's fragments. Those of
      // positions that no row sees may hold any bytes and enter as zero.
      float y0 = p0, y1 = p1, y2 = p2, y3 = p3;
      uint32_t nA = 0u, nB = 0u;
      if constexpr (ROT) {
        const uint32_t nb = rb + v_norm_offset(D, B) + 2 * (16 * ((D / 8) * g / kRotGroup) + 2 * t);
        const uint32_t ma = any >> (2 * t), mb = any >> (2 * t + 8);
        nA = lds32(nb) & ((ma & 1u ? 0xffffu : 0u) | (ma & 2u ? 0xffff0000u : 0u));
        nB = lds32(nb + 16) & ((mb & 1u ? 0xffffu : 0u) | (mb & 2u ? 0xffff0000u : 0u));
        if (mixed) {  // bits as in v0 and v1, over all groups (the lanes of a warp hold them all)
          const uint32_t bad =
              __reduce_or_sync(0xffffffffu, bad_norms(nA) << (2 * t) | bad_norms(nB) << (2 * t + 8));
          if (bad) {
            const float nan = __int_as_float(0x7fc00000);
            nA = finite_norms(nA);
            nB = finite_norms(nB);
            if (s0 && (bad >> g & 1u)) y0 = nan;
            if (s1 && (bad >> g & 1u)) y1 = nan;
            if (s2 && (bad >> (g + 8) & 1u)) y2 = nan;
            if (s3 && (bad >> (g + 8) & 1u)) y3 = nan;
          }
        }
      } else {
        const float n0 = __half2float(__ushort_as_half((unsigned short)lds16(rb + v_norm_offset(D, B) + 2 * g)));
        const float n1 = __half2float(__ushort_as_half((unsigned short)lds16(rb + v_norm_offset(D, B) + 2 * (g + 8))));
        y0 = s0 ? p0 * n0 : 0.0f;
        y1 = s1 ? p1 * n0 : 0.0f;
        y2 = s2 ? p2 * n1 : 0.0f;
        y3 = s3 ? p3 * n1 : 0.0f;
      }
      const uint32_t X0 = pack_half2(y0, y1), X1 = pack_half2(y2, y3);
      uint32_t pl[2] = {0u, 0u};
      if constexpr (C::PSPLIT) {
        const __half2 h0 = *reinterpret_cast<const __half2*>(&X0), h1 = *reinterpret_cast<const __half2*>(&X1);
        pl[0] = movmatrix_trans(pack_half2(y0 - __low2float(h0), y1 - __high2float(h0)));
        pl[1] = movmatrix_trans(pack_half2(y2 - __low2float(h1), y3 - __high2float(h1)));
      }
      pv_tile<D, B, ROT, C::PSPLIT>(rb, lut_bytes, lane4, wh, lane, movmatrix_trans(X0), movmatrix_trans(X1), pl, acc, nA, nB);
    }
    // The record is read: its stage takes the tile NSTAGE further (at two warps
    // per tile past the barrier of the exchange).
    __syncwarp();
    if constexpr (C::WT == 2) {
      if (next) xchg_get<2>(Sn, xbuf, group, (it + 1) & 1, lane);
    }
    if (leader && it + C::NSTAGE < n_iters) issue(it + C::NSTAGE);
#pragma unroll
    for (int e = 0; e < 4; ++e) S[e] = Sn[e];
  }

  // After a wait that ran out copies may still be landing: give each its bounded
  // wait before the memory is used again.
  if (leader && *(volatile int*)&s_abort)
    for (int k = n_iters > C::NSTAGE ? n_iters - C::NSTAGE : 0; k < n_iters; ++k)
      mbar_wait(&full[k % C::NSTAGE], (k / C::NSTAGE) & 1);

  // Rows that see nothing took part in the tiles that every other row sees
  // whole: they leave as empty rows.
  const bool e0 = s_row[2 * t].hi == 0, e1 = s_row[2 * t + 1].hi == 0;
  if (e0) st.m0 = -INFINITY, st.l0 = 0.0f;
  if (e1) st.m1 = -INFINITY, st.l1 = 0.0f;
#pragma unroll
  for (int i = 0; i < C::MT_W; ++i) {
    if (e0) acc[i][0] = acc[i][2] = 0.0f;
    if (e1) acc[i][1] = acc[i][3] = 0.0f;
  }
  // A NaN logit leaves the maximum alone: where it was the only one, the merges
  // must not take the row for an empty one.
  if (__any_sync(0xffffffffu, isnan(st.l0) || isnan(st.l1))) {
    float l0 = st.l0, l1 = st.l1;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    if (isnan(l0)) st.m0 = fmaxf(st.m0, 0.0f);
    if (isnan(l1)) st.m1 = fmaxf(st.m1, 0.0f);
  }
  const int64_t gid = (int64_t)(b * a.n_kv_heads + kvh) * a.n_row_groups + rg;
  const bool direct = a.n_split == 1;
  decode_epilogue<typename C::Sh, C::MT_W, ROT, true>(
      st, acc, reinterpret_cast<float*>(smem), mlbuf, group, wh, warp, lane, a.signs,
      a.part + (gid * a.n_split + split) * merge_slot_floats(D), centroid_scale(B), a.signs2, direct ? &a : nullptr, b,
      kvh, rg);
  if (direct) return;
  decode_split_tail<D, C::RING, C::THREADS, true>(a, split, gid, b, kvh, rg, threadIdx.x, smem);
}

template <int D, int B, int ROT>
static cudaError_t launch_scored_d(const ScoredArgs& a, cudaStream_t stream) {
  using C = CScored<D, B, ROT>;
  static bool configured[kMaxDevices] = {};  // the attribute is per function and device
  static ResidencyCache cap{};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !configured[dev]) {
    e = cudaFuncSetAttribute(attn_scored_kernel<D, B, ROT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) configured[dev] = true;
  }
  return launch_split_decode(attn_scored_kernel<D, B, ROT>, a, C::THREADS, C::SMEM, &cap, stream);
}

template <int D, int B, int ROT>
static cudaError_t launch_scored_any(const ScoredArgs& a, cudaStream_t stream) {
  return a.tiles ? launch_scored_tiles_d<D, B, ROT>(a, stream) : launch_scored_d<D, B, ROT>(a, stream);
}

template <int B, int ROT>
static cudaError_t launch_scored_bits(const ScoredArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64:
      if constexpr (ROT) return cudaErrorInvalidValue;
      else return launch_scored_any<64, B, 0>(a, stream);
    case 128: return launch_scored_any<128, B, ROT>(a, stream);
    case 256: return launch_scored_any<256, B, ROT>(a, stream);
    case 512: return launch_scored_any<512, B, ROT>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ckv
