// sda_append.cu -- the new tokens' rows into a paged cache, with RMSNorm and rotation on
// the way, and the same for their queries.
//
// Token i of sequence b (sda_chunk.cuh) stands at p = n_b - m_b + i; every row x of it
// becomes, in fp32,
//   y = x / sqrt(mean x^2 + eps) * w          (where weights are given)
//   (y_d, y_d+1) <- (y_d c - y_d+1 s, y_d+1 c + y_d s),  c, s = cos, sin[p][i], on the
//                                              last R dimensions
// A query is stored as bf16.  The KV row goes to its pool row, as bf16, or as E4M3 codes
// with one scale for each block of the cache: a block's new rows need
//   2^e, e least with 448 2^e >= max |y| over them (at least 2^-126, also for zeros),
// its scale becomes the larger of that and what it had (only that where it held nothing),
// and where it grows the codes that are there become e4m3(code * old / new).
//
// Layout of the work: a warp owns rows of q (and of kv into a bf16 pool), lane l their
// 16-byte chunks l, l + 32, ..., so that a pair of the rotation stays in a lane.  A warp
// takes consecutive rows, so that it looks for its sequence once, and has the next row's
// loads in flight.  8-bit blocks are CTAs of their own, ahead of the others in the grid:
// the CTA that holds a block's first new token finds its scale over all new rows of it,
// then writes them.
// What bounds it: DRAM (4 bytes an element of q), and close to it the instructions, some 250 a
// row of 512.  2048 tokens of 64 heads, D = 512, bf16 cache (273 MB): 51 us, 5.3 TB/s; with 370
// instructions a row (weights unpacked anew, registers spilled) it took 65, with places found
// anew for every row 54.  24 thousand rows without
// queries into codes: 20 us, two passes over each block's rows, 3 to 4 blocks a CTA.  Calls of few rows:
// the chain of a launch, the search for the sequence, a row's load and its store (6 us).
#include "sda_append.cuh"
#include "sda_rows.cuh"

namespace sda {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
template <int CPL, bool FP8>
constexpr int append_ctas_per_sm() { return CPL == 1 ? 4 : CPL == 2 ? 3 : 2; }

// The sequence of token t: the last b with q_indptr[b] <= t (-1: none).  128 probes a
// step, so that up to 128 sequences take one load's time.
__device__ __forceinline__ int sequence_of(const int32_t* q_indptr, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // the answer lies in [lo, lo + n), or is none
  bool none = false;
  while (n > 0) {
    const int step = (n + 127) / 128;
    int below = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = (k * 32 + lane) * step;
      below += __popc(__ballot_sync(0xffffffffu, i < n && __ldg(q_indptr + lo + min(i, n - 1)) <= t));
    }
    if (below == 0) {
      none = true;
      break;
    }
    lo += (below - 1) * step;
    n = min(step, n - (below - 1) * step);
    if (step == 1) break;
  }
  return none || B == 0 ? -1 : lo;
}

__device__ __forceinline__ void report(const AppendParams& p, int bits) {
  if (!p.one_status) atomicOr(p.status, bits);
}

// Where a warp stands: a token and its sequence.
struct Place {
  int t, b, q0, q1, n;  // sequence b: tokens q0 .. q1 - 1, n cached positions (q1 = q0: skipped)
  bool bad;
  __device__ __forceinline__ void load(const AppendParams& p) {
    q0 = __ldg(p.g.q_indptr + b);
    q1 = __ldg(p.g.q_indptr + b + 1);
    n = __ldg(p.g.kv_len + b);
    bad = lengths_bad(p.g, b);  // (the same loads)
  }
  __device__ __forceinline__ void init(const AppendParams& p, int t_) {
    t = t_;
    b = sequence_of(p.g.q_indptr, p.g.B, t);
    if (b >= 0) load(p);
  }
  // On to the next sequence, or, where that has no token behind t either, behind all that have
  // none (a padded batch may hold thousands: one by one they took 770 us); B behind the last.
  __device__ __forceinline__ void next(const AppendParams& p) {
    const int after = ++b;
    if (b >= p.g.B) return;
    load(p);
    if (t < q1) return;
    b = sequence_of(p.g.q_indptr, p.g.B, t);
    if (b <= after) b = after;
    else load(p);
  }
  // token t' > t; b = -1 before the first sequence, B behind the last
  __device__ __forceinline__ void to(const AppendParams& p, int t_) {
    t = t_;
    if (b < 0) return init(p, t_);
    while (b < p.g.B && t >= q1) next(p);
  }
  // Whether the token is one of a sequence whose lengths make sense.
  __device__ __forceinline__ bool live(const AppendParams& p) const {
    return b >= 0 && b < p.g.B && !bad && t >= q0 && t < q1;
  }
  __device__ __forceinline__ int pos() const { return n - (q1 - q0) + t - q0; }
};

__device__ __forceinline__ bool position_ok(const AppendParams& p, int pos) {
  return pos >= 0 && (p.R == 0 || pos < p.max_pos);
}

template <int CPL>
__device__ __forceinline__ void load_row(const uint16_t* src, int chunks, int lane, uint4 (&x)[CPL]) {
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    const int c = lane + 32 * j;
    x[j] = c < chunks ? __ldcs(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
  }
}

// A row's weights, 16-byte chunks as they lie in memory.
template <int CPL>
__device__ __forceinline__ void load_weights(const uint16_t* w, int chunks, int lane, uint4 (&v)[CPL]) {
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    const int c = lane + 32 * j;
    v[j] = w != nullptr && c < chunks ? __ldg(reinterpret_cast<const uint4*>(w) + c) : make_uint4(0, 0, 0, 0);
  }
}

// A row's values in place; cos_row and sin_row are its position's.  Every operation is rounded
// as in sda_store.cu, so that a row has the same bits in both stores: the mean is a division
// (inv_d: exact) and the inverse root an IEEE root and division.
template <int CPL>
__device__ __forceinline__ void row_values(const AppendParams& p, const uint4 (&w)[CPL], bool norm,
                                           const float* cos_row, const float* sin_row, int lane,
                                           float (&f)[CPL][8]) {
  const int chunks = p.g.D >> 3, chunk0 = (p.g.D - p.R) >> 3;
  if (norm) {
    uint64_t ss2 = 0;
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const uint64_t v = f2_pack(f[j][k], f[j][k + 1]);
        ss2 = f2_fma(v, v, ss2);
      }
    }
    float even, odd;
    f2_unpack(ss2, even, odd);
    float ss = even + odd;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float mean = p.inv_d != 0.f ? ss * p.inv_d : ss / (float)p.g.D;
    const float inv = 1.f / sqrtf(__fadd_rn(mean, p.eps));
    const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      float wv[8];
      unpack8(w[j], wv);
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const uint64_t y = f2_mul(f2_mul(f2_pack(f[j][k], f[j][k + 1]), inv2), f2_pack(wv[k], wv[k + 1]));
        f2_unpack(y, f[j][k], f[j][k + 1]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    const int c = lane + 32 * j;
    if (c >= chunk0 && c < chunks) {
      const float4 cs = __ldg(reinterpret_cast<const float4*>(cos_row + 4 * (c - chunk0)));
      const float4 sn = __ldg(reinterpret_cast<const float4*>(sin_row + 4 * (c - chunk0)));
      const float cv[4] = {cs.x, cs.y, cs.z, cs.w}, sv[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = f[j][2 * i], b = f[j][2 * i + 1];
        f[j][2 * i] = a * cv[i] - b * sv[i];
        f[j][2 * i + 1] = b * cv[i] + a * sv[i];
      }
    }
  }
}

__device__ __forceinline__ int block_of(const AppendParams& p, int pos) {  // pos / k_per_block
  return (int)(((unsigned long long)(unsigned)pos * p.k_mul) >> p.k_shift);
}

// Pool row of position pos of sequence b; -1 (and status bit 2): outside the pool.
__device__ __forceinline__ int64_t pool_row(const AppendParams& p, int b, int pos) {
  const int jb = block_of(p, pos);
  const int blk = __ldg(p.g.block_table + (size_t)b * p.g.max_blocks + jb);
  const int64_t row = p.g.base + (int64_t)blk * p.g.k_per_block + (pos - jb * p.g.k_per_block);
  return blk < 0 || row >= p.g.total_pages ? -1 : row;
}

// Rows of q, and of kv into a bf16 pool: `rpt` rows a token.
template <int CPL, bool FP8>
__device__ __forceinline__ void plain_rows(const AppendParams& p, int64_t worker, int64_t workers) {
  const int lane = threadIdx.x & 31, D = p.g.D, chunks = D >> 3;
  const int H = p.g.H, rpt = H + (FP8 ? 0 : 1);
  const int64_t rows = (int64_t)p.g.T * rpt, each = (rows + workers - 1) / workers;
  const int64_t r0 = worker * each;
  if (r0 >= rows) return;
  int left = (int)min(each, rows - r0), t = (int)(r0 / rpt), h = (int)(r0 - (int64_t)t * rpt);
  size_t at_q = ((size_t)t * H + h) * D;  // of the row, or of the next of q behind a row of kv
  uint4 x[CPL], wq[CPL];
  load_row<CPL>(h < H ? p.q + at_q : p.kv + (size_t)t * D, chunks, lane, x);
  load_weights<CPL>(p.q_w, chunks, lane, wq);
  const int half = p.R >> 1;
  Place at;
  at.init(p, t);
  bool live = at.live(p);
  int pos = live ? at.pos() : 0;
  bool ok = position_ok(p, pos);
  const float *cos_row = p.cos_cache + (size_t)pos * half, *sin_row = p.sin_cache + (size_t)pos * half;
  for (;; --left) {
    const bool is_kv = !FP8 && h == H;
    uint16_t* dst = p.q_out + at_q;
    if (!is_kv) at_q += D;
    int nh = h + 1;
    if (nh == rpt) nh = 0;
    float f[CPL][8];
#pragma unroll
    for (int j = 0; j < CPL; ++j) unpack8(x[j], f[j]);
    if (left > 1)
      load_row<CPL>(FP8 || nh < H ? p.q + at_q : p.kv + (size_t)(t + (nh == 0)) * D, chunks, lane, x);
    // (rows of tokens outside every sequence, or in one whose lengths make no sense, stay as they are)
    if (live) {
      if (is_kv) {
        dst = nullptr;
        if (ok) {
          const int64_t row = pool_row(p, at.b, pos);
          if (row >= 0) dst = p.pool + row * D;
          else if (lane == 0) report(p, 2);
        } else if (lane == 0) {
          report(p, 1);
        }
        uint4 wk[CPL];
        load_weights<CPL>(p.kv_w, chunks, lane, wk);
        if (dst) row_values<CPL>(p, wk, p.kv_w != nullptr, cos_row, sin_row, lane, f);
      } else if (ok) {
        row_values<CPL>(p, wq, p.q_w != nullptr, cos_row, sin_row, lane, f);
      }
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        if (dst && lane + 32 * j < chunks) {
          uint4* d4 = reinterpret_cast<uint4*>(dst) + lane + 32 * j;
          const uint4 y = ok ? pack8_bf16(f[j]) : make_uint4(0, 0, 0, 0);
          if (is_kv) *d4 = y;
          else __stcs(d4, y);
        }
      }
    }
    if (left == 1) return;
    h = nh;
    if (h == 0) {
      at.to(p, ++t);
      live = at.live(p);
      pos = live ? at.pos() : 0;
      ok = position_ok(p, pos);
      cos_row = p.cos_cache + (size_t)pos * half;
      sin_row = p.sin_cache + (size_t)pos * half;
    }
  }
}

// Rows of one block in codes: its tokens t .. t + cnt - 1 at positions pos .., in block jb of
// sequence b behind `held` rows that the block had.
template <int CPL>
__device__ __forceinline__ void block_codes(const AppendParams& p, int b, int jb, int t, int pos, int cnt, int held,
                                            float* s_max) {
  constexpr int NR = CPL <= 2 ? 2 : 1;  // rows of a warp whose loads are in flight together
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, chunks = p.g.D >> 3;
  const int K = p.g.k_per_block, half = p.R >> 1;
  uint4 x[NR][CPL], w[CPL];
  // (the first rows' loads go out before the block is looked up)
#pragma unroll
  for (int k = 0; k < NR; ++k)
    if (warp + k * kWarps < cnt) load_row<CPL>(p.kv + (size_t)(t + warp + k * kWarps) * p.g.D, chunks, lane, x[k]);
  load_weights<CPL>(p.kv_w, chunks, lane, w);
  const int blk = __ldg(p.g.block_table + (size_t)b * p.g.max_blocks + jb);
  const int64_t row0 = p.g.base + (int64_t)blk * K + held;  // of the first new row
  if (blk < 0 || row0 >= p.g.total_pages) {
    if (tid == 0) report(p, 2);
    return;
  }
  if (row0 + cnt > p.g.total_pages) {  // the block's end lies behind the pool's
    if (tid == 0) report(p, 2);
    cnt = (int)(p.g.total_pages - row0);
  }
  const float had = held > 0 ? p.scale[blk] : 0.f;
  const bool once = cnt <= NR * kWarps;  // rows stay in registers from one pass to the other
  float f[CPL][8];
  float top = 0.f;
  bool infinite = false;  // a value of this lane's
  for (int i0 = warp; i0 < cnt; i0 += NR * kWarps) {
#pragma unroll
    for (int k = 0; k < NR; ++k)
      if (i0 > warp && i0 + k * kWarps < cnt)
        load_row<CPL>(p.kv + (size_t)(t + i0 + k * kWarps) * p.g.D, chunks, lane, x[k]);
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      if (i0 + k * kWarps >= cnt) break;
      const size_t at = (size_t)(pos + i0 + k * kWarps) * half;
#pragma unroll
      for (int j = 0; j < CPL; ++j) unpack8(x[k][j], f[j]);
      row_values<CPL>(p, w, p.kv_w != nullptr, p.cos_cache + at, p.sin_cache + at, lane, f);
      float most = 0.f;  // (fmaxf passes over NaN)
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
#pragma unroll
        for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(f[j][e]));
      }
      if (most == INFINITY) {
        infinite = true;
        most = 0.f;
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
#pragma unroll
          for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(f[j][e]) < INFINITY ? fabsf(f[j][e]) : 0.f);
        }
      }
      top = fmaxf(top, most);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  __syncthreads();  // (the block before this one has been read)
  if (lane == 0) s_max[warp] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kWarps; ++k) top = fmaxf(top, s_max[k]);
  const int e = top > 0.f ? fp8_scale_exponent(top) : -126;
  const float need = __int_as_float((127 + e) << 23);
  const float s = fmaxf(had, need);  // (had NaN: need)
  if (tid == 0) p.scale[blk] = s;
  if (held > 0 && had != s) {
    // what the block held, rounded to the larger scale
    const float by = had / s;
    uint4* c = reinterpret_cast<uint4*>(p.codes + (row0 - held) * p.g.D);
    const int64_t n16 = (int64_t)held * p.g.D / 16;
    for (int64_t i = tid; i < n16; i += kThreads) c[i] = scaled_codes(c[i], by);
  }
  // (s is a power of two unless the caller's scale was none: then 1 / s is exact)
  const bool power = (__float_as_uint(s) & 0x7fffffu) == 0;
  const float inv = 1.f / s;
  for (int i0 = warp; i0 < cnt; i0 += NR * kWarps) {
    if (!once) {
#pragma unroll
      for (int k = 0; k < NR; ++k)
        if (i0 + k * kWarps < cnt)
          load_row<CPL>(p.kv + (size_t)(t + i0 + k * kWarps) * p.g.D, chunks, lane, x[k]);
    }
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      const int i = i0 + k * kWarps;
      if (i >= cnt) break;
      const size_t at = (size_t)(pos + i) * half;
#pragma unroll
      for (int j = 0; j < CPL; ++j) unpack8(x[k][j], f[j]);
      row_values<CPL>(p, w, p.kv_w != nullptr, p.cos_cache + at, p.sin_cache + at, lane, f);
      uint2* dst = reinterpret_cast<uint2*>(p.codes + (row0 + i) * p.g.D);
      if (power) {
        const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
#pragma unroll
          for (int v = 0; v < 8; v += 2) f2_unpack(f2_mul(f2_pack(f[j][v], f[j][v + 1]), inv2), f[j][v], f[j][v + 1]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
#pragma unroll
          for (int v = 0; v < 8; ++v) f[j][v] = __fdiv_rn(f[j][v], s);
        }
      }
      if (infinite) {
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            if (fabsf(f[j][v]) == INFINITY) f[j][v] = NAN;  // E4M3 has no infinity
          }
        }
      }
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        if (lane + 32 * j < chunks) dst[lane + 32 * j] = pack8_e4m3(f[j]);
      }
    }
  }
}

// The blocks whose first new token lies in [t, t1).
template <int CPL>
__device__ __forceinline__ void code_blocks(const AppendParams& p, int t, int t1, float* s_max) {
  const int K = p.g.k_per_block;
  // The rows come to L2 while the sequence is looked for.
  const char* rows = reinterpret_cast<const char*>(p.kv + (size_t)t * p.g.D);
  for (int64_t o = threadIdx.x * 128; o < (int64_t)(t1 - t) * p.g.D * 2; o += kThreads * 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(rows + o));
  Place at;
  at.init(p, t);
  if (at.b < 0) {  // before the first sequence
    at.b = 0;
    at.load(p);
    at.t = max(t, at.q0);
  }
  while (at.t < t1 && at.b < p.g.B) {
    if (at.bad || at.t >= at.q1) {
      at.next(p);
      if (at.b < p.g.B) at.t = max(at.t, at.q0);
      continue;
    }
    int pos = at.pos();
    const int end = p.R == 0 ? at.n : min(at.n, p.max_pos);
    if (threadIdx.x == 0 && at.t == at.q0 && (pos < 0 || end < at.n)) report(p, 1);
    // to the next token that is its block's first (position 0, where there are more
    // tokens than positions)
    int jb = block_of(p, max(pos, 0)), in = max(pos, 0) - jb * K;  // block, and row in it
    int skip = pos < 0 ? -pos : (at.t == at.q0 || in == 0 ? 0 : K - in);
    if (pos >= 0 && skip > 0) ++jb, in = 0;
    skip = min(skip, at.q1 - at.t);
    at.t += skip;
    pos += skip;
    if (at.t >= at.q1 || at.t >= t1) continue;
    const int cnt = min(min(at.q1 - at.t, K - in), end - pos);
    if (cnt > 0) block_codes<CPL>(p, at.b, jb, at.t, pos, cnt, in, s_max);
    ++at.t;
  }
}

// The status word by one CTA, for calls of few sequences and blocks: a sequence a thread, and the
// blocks of one that writes many by its warp.
__device__ __forceinline__ void whole_status(const AppendParams& p) {
  const int K = p.g.k_per_block, lane = threadIdx.x & 31;
  int bits = 0;
  auto look = [&](int b, int jb, int end) {  // at the block's last row
    const int blk = __ldg(p.g.block_table + (size_t)b * p.g.max_blocks + jb);
    const int last = (int)min((long long)K, (long long)end - (long long)jb * K) - 1;
    return blk < 0 || p.g.base + (int64_t)blk * K + last >= p.g.total_pages ? 2 : 0;
  };
  for (int b0 = (int)threadIdx.x - lane; b0 < p.g.B; b0 += kThreads) {
    const int b = b0 + lane;
    int first = 0, last = -1, end = 0;  // blocks that are written
    if (b < p.g.B) {
      if (lengths_bad(p.g, b)) {
        bits |= 4;
      } else {
        const int m = __ldg(p.g.q_indptr + b + 1) - __ldg(p.g.q_indptr + b), n = __ldg(p.g.kv_len + b);
        end = p.R == 0 ? n : min(n, p.max_pos);
        if (m > 0 && (n < m || end < n)) bits |= 1;
        const int from = max(n - m, 0);
        if (m > 0 && from < end) {
          first = block_of(p, from);
          last = block_of(p, end - 1);
        }
      }
    }
    if (last - first < 2) {
      for (int jb = first; jb <= last; ++jb) bits |= look(b, jb, end);
    }
    for (uint32_t many = __ballot_sync(0xffffffffu, last - first >= 2); many; many &= many - 1) {
      const int l = __ffs(many) - 1, f = __shfl_sync(0xffffffffu, first, l), t = __shfl_sync(0xffffffffu, last, l);
      const int e = __shfl_sync(0xffffffffu, end, l);
#pragma unroll 4
      for (int jb = f + lane; jb <= t; jb += 32) bits |= look(b0 + l, jb, e);
    }
  }
  const int any1 = __syncthreads_or(bits & 1), any2 = __syncthreads_or(bits & 2), any4 = __syncthreads_or(bits & 4);
  if (threadIdx.x == 0) *p.status = (any1 ? 1 : 0) | (any2 ? 2 : 0) | (any4 ? 4 : 0);
}

template <int CPL, bool FP8>
__global__ void __launch_bounds__(kThreads, append_ctas_per_sm<CPL, FP8>()) append_kernel(const AppendParams p) {
  __shared__ float s_max[kWarps];
  pdl_wait();
  pdl_trigger();
  const int before = p.one_status ? 1 : 0;
  if ((int)blockIdx.x < before) return whole_status(p);
  const int cta = (int)blockIdx.x - before - p.code_ctas;
  if constexpr (FP8) {
    if (cta < 0) {
      const int64_t t = (int64_t)((int)blockIdx.x - before) * p.code_tokens;
      code_blocks<CPL>(p, (int)t, (int)min(t + p.code_tokens, (int64_t)p.g.T), s_max);
    }
  }
  if (!FP8 || cta >= 0)
    plain_rows<CPL, FP8>(p, (int64_t)cta * kWarps + (threadIdx.x >> 5),
                         (int64_t)((int)gridDim.x - before - p.code_ctas) * kWarps);
  if (p.one_status) return;
  // lengths that make no sense, of sequences without tokens too
  for (int64_t b = (int64_t)blockIdx.x * kThreads + threadIdx.x; b < p.g.B; b += (int64_t)gridDim.x * kThreads)
    if (lengths_bad(p.g, (int)b)) atomicOr(p.status, 4);
}

template <int CPL, bool FP8>
cudaError_t launch(AppendParams& p, int num_sms, cudaStream_t st) {
  const int64_t resident = (int64_t)num_sms * append_ctas_per_sm<CPL, FP8>();
  const int64_t rows = (int64_t)p.g.T * (p.g.H + (FP8 ? 0 : 1));
  const int64_t row_ctas = std::min((rows + kWarps - 1) / kWarps, resident - (p.one_status ? 1 : 0));
  p.code_ctas = 0;
  division(p.g.k_per_block, &p.k_mul, &p.k_shift);
  if (FP8) {
    // tokens to a CTA: one where there are few; CTAs that come later would look for their
    // sequence anew
    p.code_tokens = (int)((p.g.T + resident - 1) / resident);
    p.code_ctas = (p.g.T + p.code_tokens - 1) / p.code_tokens;
  }
  return launch_pdl(append_kernel<CPL, FP8>, dim3((unsigned)(row_ctas + p.code_ctas + (p.one_status ? 1 : 0))), dim3(kThreads), 0, st,
                    (const AppendParams&)p);
}

}  // namespace

// Whether one CTA looks at all that the status word tells of, in place of a clear of the word
// (a launch of its own) and atomics of whoever finds something: for some thousand loads
// that take a few microseconds together.  A step of 64 sequences, replayed: 6.3 us with it, 8.3
// without; 2048 tokens of 64 heads 51.6 us, 53.4 without.
bool append_one_status(const AppendParams& p) {
  // (blocks of many rows take longer to write than to look at)
  return p.g.B <= kThreads && p.g.T / p.g.k_per_block <= (p.g.k_per_block >= 16 ? 2048 : 512);
}

cudaError_t launch_append(AppendParams p, int num_sms, cudaStream_t st) {
  const bool fp8 = p.codes != nullptr;
  const int cpl = (p.g.D / 8 + 31) / 32;
#define SDA_APPEND(C) return fp8 ? launch<C, true>(p, num_sms, st) : launch<C, false>(p, num_sms, st)
  if (cpl <= 1) SDA_APPEND(1);
  if (cpl <= 2) SDA_APPEND(2);
  SDA_APPEND(4);
#undef SDA_APPEND
}

}  // namespace sda
