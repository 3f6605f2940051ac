// tree_accept.cu — the accepted path of a drafted tree, moved inside the packed
// cache: position base + path[j] goes to base + j, bit for bit.
//
// A position is not a run of bytes: its K codes are 8-byte chunks of a record
// and its V codes are fields in words that it shares with the record's other
// positions. One CTA owns a (sequence, kv head), a warp one accepted node at a
// time: every warp first reads its nodes' parts into registers, then, past one
// barrier, all of them write, so the order of the path and sources that are
// also targets do not matter. The writes of shared words commute (each
// position clears and sets its own bits). Nothing to compute and a few
// kilobytes to move per CTA: the time is the launch and two dependent trips to
// memory (the lengths and the path, then the rows).
#include "ckv_kernels.cuh"
#include "pack_common.cuh"

namespace ckv {

namespace {

constexpr int kAcceptWarps = 16, kAcceptPath = 64, kAcceptPer = kAcceptPath / kAcceptWarps;

// The window of lane `lane`'s V bits of position p: lane stream, first word,
// shift, and (with the bits' compact form, the same for every position) the
// words' masks.
template <int D, int B>
struct VWindow {
  static constexpr int E = D / 32;
  static constexpr int NW = pack::PositionCodes<D, B>::NW;
  int L, w0, sh;
  __device__ __forceinline__ VWindow(int p, int lane) {
    L = 4 * (lane >> 2) + ((p & 7) >> 1);
    const int start = 4 * B * E * (lane & 3) + 4 * B * (p >> 3) + B * (p & 1);
    w0 = start >> 5;
    sh = start & 31;
  }
  // Compact bits [8B (e / 2) + 2B (e % 2), + B) of values e < E.
  static __device__ __forceinline__ uint32_t compact_mask(int w) {
    uint32_t m = 0u;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const int bit = 8 * B * (e >> 1) + 2 * B * (e & 1) + k;
        if (bit >> 5 == w) m |= 1u << (bit & 31);
      }
    return m;
  }
  __device__ __forceinline__ uint32_t mask(int w) const {
    return __funnelshift_l(w > 0 ? compact_mask(w - 1) : 0u, compact_mask(w), sh);
  }
};

// One position's parts, a lane's share; V bits in compact form.
template <int D, int B>
struct MovedPosition {
  static constexpr int E = D / 32, NW = VWindow<D, B>::NW;
  uint32_t q[(E + 3) / 4];
  __half d16, n16;
  uint32_t v[NW];
};

template <int D, int B, int ROT>
__device__ __forceinline__ void read_position(const uint8_t* rec, int p, int lane, MovedPosition<D, B>& m) {
  constexpr int E = D / 32, LPB = 32 / E;
  if constexpr (E >= 8) {
#pragma unroll
    for (int c = 0; c < E / 8; ++c) {
      const uint2 w = *reinterpret_cast<const uint2*>(rec + pack::k_chunk_byte(p, E * lane / 8 + c));
      m.q[2 * c] = w.x;
      m.q[2 * c + 1] = w.y;
    }
  } else {
    const uint8_t* src = rec + pack::k_chunk_byte(p, E * lane / 8) + (E * lane) % 8;
    if constexpr (E == 4) m.q[0] = *reinterpret_cast<const uint32_t*>(src);
    else m.q[0] = *reinterpret_cast<const uint16_t*>(src);
  }
  m.d16 = *reinterpret_cast<const __half*>(rec + k_scale_offset(D) + 2 * (p * (D / 32) + lane / LPB));
  const int grp = ROT ? lane / (kRotGroup / E) : 0;
  m.n16 = *reinterpret_cast<const __half*>(rec + v_norm_offset(D, B) + 2 * (16 * grp + p));
  const VWindow<D, B> win(p, lane);
  uint32_t x[VWindow<D, B>::NW + 1];
#pragma unroll
  for (int w = 0; w < VWindow<D, B>::NW; ++w)  // words outside the stream carry none of the position's bits
    x[w] = win.mask(w) ? *reinterpret_cast<const uint32_t*>(rec + pack::v_word_offset<D, B>(win.L, win.w0 + w)) : 0u;
  x[VWindow<D, B>::NW] = 0u;
#pragma unroll
  for (int w = 0; w < VWindow<D, B>::NW; ++w)
    m.v[w] = __funnelshift_r(x[w], x[w + 1], win.sh) & VWindow<D, B>::compact_mask(w);
}

template <int D, int B, int ROT>
__device__ __forceinline__ void write_position(uint8_t* rec, int p, int lane, const MovedPosition<D, B>& m) {
  constexpr int E = D / 32, LPB = 32 / E;
  pack::PositionCodes<D, B> pc;
#pragma unroll
  for (int e = 0; e < E; ++e) pc.q[e] = static_cast<uint8_t>(m.q[e / 4] >> (8 * (e % 4)));
  pack::store_k_codes<E>(rec, p, lane, pc.q);
  if (lane % LPB == 0)
    *reinterpret_cast<__half*>(rec + k_scale_offset(D) + 2 * (p * (D / 32) + lane / LPB)) = m.d16;
  pack::store_norm<D, B, ROT>(rec, p, lane, m.n16);
  const VWindow<D, B> win(p, lane);
#pragma unroll
  for (int w = 0; w < VWindow<D, B>::NW; ++w) {
    const uint32_t mask = win.mask(w);
    if (mask) {
      uint32_t* word = reinterpret_cast<uint32_t*>(rec + pack::v_word_offset<D, B>(win.L, win.w0 + w));
      atomicAnd(word, ~mask);
      atomicOr(word, __funnelshift_l(w > 0 ? m.v[w - 1] : 0u, m.v[w], win.sh));
    }
  }
}

template <int D, int B, int ROT>
__global__ void __launch_bounds__(kAcceptWarps * 32) tree_accept_kernel(AcceptArgs a) {
  constexpr int REC = record_bytes(D, B, ROT ? D / kRotGroup : 1);
  const int h = blockIdx.x, b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_warps = blockDim.x >> 5;
  griddep_wait();
  const int T = a.seq_len[b], n = a.q_len ? a.q_len[b] : a.n_q, count = a.path_len[b];
  const int32_t* path = a.path + (int64_t)b * a.max_path;
  bool bad = T < 0 || T > a.capacity || n < 0 || n > a.n_q || n > T || count < 0 || count > a.max_path;
  int p0 = 0, p1 = 0;  // path[lane], path[lane + 32]: every warp checks the whole path
  if (!bad) {
    p0 = lane < count ? path[lane] : 0;
    p1 = lane + 32 < count ? path[lane + 32] : 0;
    const bool out = (lane < count && (p0 < 0 || p0 >= n)) || (lane + 32 < count && (p1 < 0 || p1 >= n));
    bad = __any_sync(0xffffffffu, out);
  }
  const int base = T - n;
  if (h == 0 && threadIdx.x == 0) {
    a.new_len[b] = bad ? T : base + count;
    if (bad) raise_flag(a.flag, kFlagSeqLenRange);
  }
  if (bad) return;
  uint8_t* stream = a.cache + ((int64_t)b * a.n_kv_heads + h) * (a.capacity / kTile) * REC;
  MovedPosition<D, B> m[kAcceptPer];
  auto each = [&](auto&& f) {  // f(slot, target, source) for this warp's nodes that move
#pragma unroll
    for (int k = 0; k < kAcceptPer; ++k) {
      const int j = warp + k * n_warps;
      const int s = __shfl_sync(0xffffffffu, j < 32 ? p0 : p1, j & 31);
      if (j < count && s != j) f(m[k], base + j, base + s);
    }
  };
  each([&](MovedPosition<D, B>& x, int, int from) {
    read_position<D, B, ROT>(stream + (int64_t)(from / kTile) * REC, from % kTile, lane, x);
  });
  __syncthreads();
  each([&](MovedPosition<D, B>& x, int to, int) {
    write_position<D, B, ROT>(stream + (int64_t)(to / kTile) * REC, to % kTile, lane, x);
  });
}

template <int D, int B, int ROT>
static cudaError_t launch_accept_dbr(const AcceptArgs& a, cudaStream_t stream) {
  // Enough warps that no warp has more than kAcceptPer nodes.
  const int warps = a.max_path < kAcceptWarps ? a.max_path : kAcceptWarps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.n_kv_heads, a.batch);
  cfg.blockDim = dim3(32 * warps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_accept_kernel<D, B, ROT>, a);
}

template <int D, int B>
static cudaError_t launch_accept_db(const AcceptArgs& a, cudaStream_t stream) {
  if constexpr (D >= kRotGroup) {
    if (a.rot) return launch_accept_dbr<D, B, 1>(a, stream);
  } else {
    if (a.rot) return cudaErrorInvalidValue;
  }
  return launch_accept_dbr<D, B, 0>(a, stream);
}

template <int D>
static cudaError_t launch_accept_d(const AcceptArgs& a, cudaStream_t stream) {
  switch (a.v_bits) {
    case 2: return launch_accept_db<D, 2>(a, stream);
    case 3: return launch_accept_db<D, 3>(a, stream);
    case 4: return launch_accept_db<D, 4>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_tree_accept(const AcceptArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return launch_accept_d<64>(a, stream);
    case 128: return launch_accept_d<128>(a, stream);
    case 256: return launch_accept_d<256>(a, stream);
    case 512: return launch_accept_d<512>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace ckv
