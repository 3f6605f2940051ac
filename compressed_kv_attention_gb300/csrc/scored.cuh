// scored.cuh — what attn_scored and attn_tree add to attention over the packed
// cache: per-row visibility (causal rows, sliding window, document and prefix
// masks, or a drafted tree's ancestor masks), the tanh cap and the distance bias.
//
// Row (token i of the n newest positions of a sequence of length T; n = q_len
// or n_q, base = T - n):
//   causal rows: at = base + i, sees p in [max(doc, at - window + 1, 0),
//                max(at + 1, min(prefix, T)))
//   tree rows:   mask m_i, at = base + popcount(m_i) - 1 (the depth); sees
//                p < base with p > at - window, and node j (position base + j)
//                where bit j of m_i is set and at - at_j < window
// Logit: x = c tanh(scale q.k / c) - slope |at - at_key|, in log2 units here.
#pragma once

#include "ckv_kernels.cuh"

namespace ckv {

struct ScoredArgs : DecodeArgs {
  const int32_t* q_len;      // query tokens per sequence (the rows after them are empty) or nullptr: n_q
  const uint64_t* tree;      // [batch][n_q] ancestor masks (attn_tree) or nullptr
  const float* slopes;       // [n_q_heads] or nullptr
  const int32_t* prefix_len; // [batch] or nullptr
  const int32_t* doc_start;  // [batch][n_q] or nullptr
  int window;                // 0: none
  // The tcgen05 form (128 query rows per CTA): n_split shares of each tile's
  // keys, partial rows at part ([tile][split][128][D + 1]: normalised rotated
  // rows, then their lse) when there are several.
  int tiles;
  // Without a cap (cap_log2 0) the logit is mul * S; with one it is
  // cap_log2 * tanh(mul * S).
  float mul, cap_log2;
};

// One query row: the interval [lo, hi) of its keys (empty: lo = hi = 0), its
// position, its slope in log2 units, and (trees) its drafted keys' bits.
struct RowInfo {
  int lo, hi, at;
  float slope;
  uint64_t tree;
};

__device__ __forceinline__ uint64_t low_bits(int n) { return n >= 64 ? ~0ull : (1ull << n) - 1ull; }

// Tokens of sequence b that are queries, and the length the rows see; both 0
// (every row empty, the device flag raised by `raise`) when out of range. A
// sequence shorter than its queries is legal for causal rows (the rows before
// its first position are empty) and not for a tree.
__device__ __forceinline__ void scored_lengths(const ScoredArgs& a, int b, bool raise, int& seqlen, int& n) {
  const int64_t lim = a.capacity < a.max_seq_len ? a.capacity : a.max_seq_len;
  seqlen = a.seq_len[b];
  n = a.q_len ? a.q_len[b] : a.n_q;
  const bool bad = seqlen < 0 || seqlen > lim || n < 0 || n > a.n_q || (a.tree && n > seqlen);
  if (bad) {
    if (raise) raise_flag(a.flag, kFlagSeqLenRange);
    seqlen = n = 0;
  }
}

// Everything a row reads from memory, issued at once (beside the lengths).
struct RowLoads {
  float slope;
  int prefix, doc;
  uint64_t tree;
};
__device__ __forceinline__ RowLoads scored_row_loads(const ScoredArgs& a, int b, int kvh, int rr) {
  const int G = a.n_q_heads / a.n_kv_heads, i = rr / G;
  RowLoads l{0.0f, 0, 0, 0ull};
  if (i >= a.n_q) return l;
  if (a.slopes) l.slope = a.slopes[kvh * G + rr % G] * 1.4426950408889634f;
  if (a.prefix_len) l.prefix = a.prefix_len[b];
  if (a.doc_start) l.doc = a.doc_start[(int64_t)b * a.n_q + i];
  if (a.tree) l.tree = a.tree[(int64_t)b * a.n_q + i];
  return l;
}

__device__ __forceinline__ RowInfo scored_row(const ScoredArgs& a, int b, int rr, const RowLoads& in, int seqlen,
                                              int n) {
  RowInfo r{0, 0, 0, 0.0f, 0ull};
  const int i = rr / (a.n_q_heads / a.n_kv_heads);
  if (i >= n) return r;
  r.slope = in.slope;
  const int base = seqlen - n;
  int64_t lo = 0;
  if (a.tree) {
    r.tree = in.tree & low_bits(n);
    const int depth = __popcll(r.tree) - 1;
    r.at = base + depth;
    r.hi = seqlen;
    if (a.window) {
      lo = (int64_t)r.at - a.window + 1;
      if (a.window < 64) {  // drafted keys further above than the window (depths differ by 63 at most)
        const uint64_t* masks = a.tree + (int64_t)b * a.n_q;
        for (int j = 0; j < n; ++j)
          if ((r.tree >> j & 1ull) && depth - (__popcll(masks[j] & low_bits(n)) - 1) >= a.window)
            r.tree &= ~(1ull << j);
      }
    }
    // The interval bounds the committed keys only: the drafted ones are the bits.
    lo = min(lo, (int64_t)base);
  } else {
    r.at = base + i;
    if (r.at < 0) return RowInfo{0, 0, 0, 0.0f, 0ull};
    r.hi = r.at + 1;
    if (a.prefix_len) r.hi = max(r.hi, min(in.prefix, seqlen));
    if (a.window) lo = (int64_t)r.at - a.window + 1;
    if (a.doc_start) lo = max(lo, (int64_t)in.doc);
  }
  r.lo = static_cast<int>(min(max(lo, (int64_t)0), (int64_t)r.hi));
  if (r.lo >= r.hi || (a.tree && r.lo == base && r.tree == 0ull)) r.lo = r.hi = 0;
  return r;
}

// Which of the 16 positions from tpos on a row sees, bit k for tpos + k.
__device__ __forceinline__ uint32_t scored_tile_bits(const RowInfo& r, bool tree, int base, int64_t tpos) {
  const int64_t l = r.lo - tpos, h = r.hi - tpos;
  if (h <= 0 || l >= 16) return 0u;
  uint32_t m = h >= 16 ? 0xffffu : (1u << h) - 1u;
  if (l > 0) m &= ~((1u << l) - 1u);
  if (tree) {
    const int64_t off = tpos - base;
    if (off >= 0) {
      m &= off < 64 ? static_cast<uint32_t>(r.tree >> off) : 0u;
    } else if (off > -16) {
      const int before = static_cast<int>(-off);  // committed keys of this tile
      m &= static_cast<uint32_t>(r.tree << before) | ((1u << before) - 1u);
    }
  }
  return m;
}

// The same for the 64 positions from tpos on.
__device__ __forceinline__ uint64_t scored_step_bits(const RowInfo& r, bool tree, int base, int64_t tpos) {
  const int64_t l = r.lo - tpos, h = r.hi - tpos;
  if (h <= 0 || l >= 64) return 0ull;
  uint64_t m = h >= 64 ? ~0ull : (1ull << h) - 1ull;
  if (l > 0) m &= ~((1ull << l) - 1ull);
  if (tree) {
    const int64_t off = tpos - base;
    if (off >= 0) {
      m &= off < 64 ? r.tree >> off : 0ull;
    } else if (off > -64) {
      const int before = static_cast<int>(-off);
      m &= (r.tree << before) | ((1ull << before) - 1ull);
    }
  }
  return m;
}

// Stored norms that are not finite (V rows beyond fp16, NaN in V). In the
// rotated tiers the norms scale V, which all rows share, and 0 times such a
// norm would reach rows that do not see the position: where some rows see it and
// some do not, it leaves V and the rows that see it get NaN through P'.
// finite_norms: a pair of norms, those that are not finite as zero; bad_norms:
// bit 0 (low) and bit 1 (high) of the pair set where it is not finite.
__device__ __forceinline__ uint32_t bad_norms(uint32_t pair) {
  const uint32_t t = (pair & 0x7c007c00u) + 0x04000400u;
  return (t >> 15 & 1u) | (t >> 30 & 2u);
}
__device__ __forceinline__ uint32_t finite_norms(uint32_t pair) {
  const uint32_t t = ((pair & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
  return pair & ~((t >> 15) * 0xffffu);
}

// tanh to about 4 units in the last place: x (1 - x^2/3 + 2 x^4/15 -
// 17 x^6/315), its Taylor series, below 1/4 (the next term is 3e-7 of the
// value there), else 1 - 2 / (1 + e^(2|x|)); the hardware's approximate tanh
// is good to 2^-11 only, 0.02 in a logit capped at 50.
__device__ __forceinline__ float tanh_f32(float x) {
  const float ax = fabsf(x), x2 = x * x;
  const float small = x * fmaf(x2, fmaf(x2, fmaf(x2, -17.0f / 315.0f, 2.0f / 15.0f), -1.0f / 3.0f), 1.0f);
  const float big = copysignf(1.0f - __fdividef(2.0f, 1.0f + fast_exp2(fminf(ax * 2.8853900817779268f, 100.0f))), x);
  return ax < 0.25f ? small : big;
}

// 1 - 2 / (1 + e^(2x)) alone: exact to about 4e-7 absolute, not relative, which
// is all a logit needs while the cap is small: at caps up to 100 (kShortCap, in
// log2 units) the logit is within 6e-5, and the probabilities within the
// rounding of their fp16 form.
constexpr float kShortCap = 144.3f;
__device__ __forceinline__ float tanh_short(float x) {
  return fmaf(-2.0f, fast_rcp(1.0f + fast_exp2(x * 2.8853900817779268f)), 1.0f);
}

// The row's logit for one raw product S, before its mask.
__device__ __forceinline__ float scored_logit(float s, float mul, float cap_log2) {
  return cap_log2 == 0.0f        ? s * mul
         : cap_log2 <= kShortCap ? cap_log2 * tanh_short(s * mul)
                                 : cap_log2 * tanh_f32(s * mul);
}

// Position of a key for the distance bias: a drafted key counts by its depth.
__device__ __forceinline__ int scored_key_at(const int8_t* depth, bool tree, int base, int p) {
  return tree && p >= base && p < base + 64 ? base + depth[p - base] : p;
}

// The depth of every drafted node of sequence b (threads tid < 64).
__device__ __forceinline__ void scored_depths(const ScoredArgs& a, int b, int n, int tid, int8_t* depth) {
  if (a.tree && tid < 64)
    depth[tid] = tid < n ? static_cast<int8_t>(__popcll(a.tree[(int64_t)b * a.n_q + tid] & low_bits(n)) - 1) : 0;
}

// One translation unit per tier (bits per V code) and rotation.
cudaError_t launch_scored_tbq2(const ScoredArgs& a, cudaStream_t stream);
cudaError_t launch_scored_tbq3(const ScoredArgs& a, cudaStream_t stream);
cudaError_t launch_scored_tbq4(const ScoredArgs& a, cudaStream_t stream);
cudaError_t launch_scored_rot2(const ScoredArgs& a, cudaStream_t stream);
cudaError_t launch_scored_rot3(const ScoredArgs& a, cudaStream_t stream);
cudaError_t launch_scored_rot4(const ScoredArgs& a, cudaStream_t stream);

}  // namespace ckv
