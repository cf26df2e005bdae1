// A K/V cache held in 4 bits: appending to it, reading it back, attention of
// one token per sequence over it, and its eviction by accumulated attention
// weight.  Part of attn_fwd.cu (same PTX wrappers, same launch helpers).
//
// Format.  The cache of one (batch b, key head h) is `cap` slots.  Each slot
// holds a K row and a V row of D channels; every 64 channels share a scale s
// and a minimum m (both bf16), and each value is a code c in 0 .. 15 that
// stands for c*s + m:
//     m = bf16(min x),  s = bf16((max x - min x) / 15),
//     c = clamp(rint((x - m) / s), 0, 15)   (0 where s is 0).
// Channel 2i of a row is the low half of byte i, channel 2i + 1 the high half.
// That is 4.5 bits a value.  A row stays whole in D/2 consecutive bytes, so
// eviction moves rows and nothing is ever requantised.  A group that holds a
// value that is not finite gets s = m = NaN.

namespace {

constexpr int kC4Group = 64;       // channels that share a scale and a minimum
constexpr unsigned kC4Overflow = 4u;  // g_attn_status: entries beyond the capacity were dropped

struct Cache4 {
  uint8_t* k;        // [B][H][cap][D/2]
  uint8_t* v;
  uint32_t* km;      // [B][H][cap][D/64], bf16 (s, m): s in the low half
  uint32_t* vm;
  int H;
  int cap;
};

// Number of cache entries of sequence b that a call sees.
__device__ __forceinline__ int c4_len(const int32_t* __restrict__ len, int b, int most) {
  return min(max(__ldg(len + b), 0), most);
}

struct Cache4Rows {
  const int32_t* seq_start;  // [B + 1], or null: row b belongs to sequence b
  const int32_t* slot0;      // [B] first slot of each sequence's rows, or null: 0
  int B;
  int64_t rows;
  int64_t k_stride, v_stride;  // elements from one packed row to the next
};

// Start of sequence b among the rows there are: what seq_start says outside of
// them counts for nothing.
__device__ __forceinline__ int c4_start(const Cache4Rows& g, int b) {
  return static_cast<int>(min(max(static_cast<int64_t>(__ldg(g.seq_start + b)), static_cast<int64_t>(0)), g.rows));
}
// Rows of sequence b.
__device__ __forceinline__ int c4_rows_of(const Cache4Rows& g, int b) {
  return g.seq_start != nullptr ? max(0, c4_start(g, b + 1) - c4_start(g, b)) : 1;
}

// The sequence that packed row `row` belongs to: the last b with start[b] <=
// row (sequences of no rows are stepped over), or B when row lies behind them
// all or before the first.
__device__ __forceinline__ int c4_sequence(const Cache4Rows& g, int row) {
  if (row < c4_start(g, 0) || row >= c4_start(g, g.B)) return g.B;
  int lo = 0, hi = g.B;  // start[lo] <= row < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (c4_start(g, mid) <= row)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Blocks of kC4RowsThreads threads; 8 channels (one 4-byte word of codes) a
// thread.  A block takes 16 (D = 128) or 32 (D = 64) packed rows and walks a run
// of their key heads, so the search for a row's sequence is made once; few rows
// are spread over more blocks by shorter runs.
constexpr int kC4RowsThreads = 256;
template <int D>
constexpr int kC4RowLanes = D / 8;
template <int D>
constexpr int kC4BlockRows = kC4RowsThreads / kC4RowLanes<D>;

// This thread's row: where it goes in the first key head's entries (b*H*cap +
// slot, -1 for nothing to do), sequence, and number among the sequence's rows.
struct C4Row {
  int64_t at;
  int b, i;
  bool dropped;  // a row of a sequence, but of no slot there is
};
// kAppend: slot0 is the cache's length, which counts as 0 where it is negative.
template <bool kAppend>
__device__ __forceinline__ C4Row c4_row(const Cache4Rows& g, const Cache4& c, int64_t row) {
  C4Row r{-1, 0, 0, false};
  if (row >= g.rows) return r;
  r.b = static_cast<int>(row);
  if (g.seq_start != nullptr) {
    r.b = c4_sequence(g, static_cast<int>(row));
    if (r.b >= g.B) return r;
    r.i = static_cast<int>(row) - c4_start(g, r.b);
  }
  int slot0 = g.slot0 != nullptr ? __ldg(g.slot0 + r.b) : 0;
  if (kAppend) slot0 = max(slot0, 0);
  const int64_t slot = static_cast<int64_t>(slot0) + r.i;
  r.dropped = slot < 0 || slot >= c.cap;
  if (!r.dropped) r.at = static_cast<int64_t>(r.b) * c.H * c.cap + slot;
  return r;
}

// Packed 16-bit minimum and maximum that pass a NaN on.
template <int kType>
__device__ __forceinline__ uint32_t min_16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (kType == kFP16)
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <int kType>
__device__ __forceinline__ uint32_t max_16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (kType == kFP16)
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// (w & mask) | magic in one instruction.  Left to the compiler it became two,
// and these are the attention kernel's most frequent ones: its ALU instructions
// for 16 keys at D = 128 went from 228 to 170 with it.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(magic));
  return r;
}
// Two fp32 operations in one instruction, each rounded as the single one.
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// One row's 8 channels of this thread (packed): the group's statistics over
// its 8 lanes, the codes and the (s, m) word.
//
// The codes are those of IEEE subtraction and division.  With y the correctly
// rounded 1 / s and q0 = d * y, q0 + (d - q0 * s) * y, each step a fused
// multiply-add, is the correctly rounded d / s (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990), as long
// as nothing under- or overflows: s within 2^-100 .. 2^100, else the division
// itself is used (a group of such values alone pays for it), on halves where the
// values are large: max - min may be twice what fp32 holds, 15 times s is not.
template <int kType>
__device__ __forceinline__ uint32_t c4_quantise(const uint4& raw, uint32_t* meta) {
  const uint32_t lo2 = min_16x2<kType>(min_16x2<kType>(raw.x, raw.y), min_16x2<kType>(raw.z, raw.w));
  const uint32_t hi2 = max_16x2<kType>(max_16x2<kType>(raw.x, raw.y), max_16x2<kType>(raw.z, raw.w)) ^ 0x80008000u;
  // (minimum, -maximum) in one register: one shuffle and one minimum for both
  uint32_t both = min_16x2<kType>(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) both = min_16x2<kType>(both, __shfl_xor_sync(0xffffffffu, both, off));
  const float2 ends = unpack_16x2<kType>(both);
  const float lo = ends.x, hi = -ends.y;
  if (!(lo > -INFINITY && hi < INFINITY)) {  // also where either is NaN
    *meta = 0x7fc07fc0u;                     // (NaN, NaN)
    return 0u;
  }
  const float range = __fsub_rn(hi, lo);
  constexpr float kFifteenth = 1.f / 15.f;
  const float q0 = __fmul_rn(range, kFifteenth);
  uint32_t sm = pack_bf16x2(__fmaf_rn(__fmaf_rn(-q0, 15.f, range), kFifteenth, q0), lo);
  float s = bf16_lo(sm);
  const float m = bf16_hi(sm);
  uint64_t x[4];  // x - m
  const uint64_t minus_m = pack_f32x2(-m, -m);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = unpack_16x2<kType>((&raw.x)[e]);
    x[e] = add_f32x2(pack_f32x2(f.x, f.y), minus_m);
  }
  uint32_t w = 0u;
  if (s >= 0x1p-100f && s <= 0x1p100f) {
    const float y1 = __frcp_rn(s);
    const uint64_t y = pack_f32x2(y1, y1), minus_s = pack_f32x2(-s, -s), magic = pack_f32x2(12582912.f, 12582912.f);
    // Rounding half to even by adding 1.5 * 2^23 leaves the code in the low bits
    // of a constant, which comes off the packed word once.
    // m is min x itself for bf16, so d / s lies within 0 .. 15.06; fp16's
    // minimum is rounded to bf16, so there it may fall outside.
#pragma unroll
    for (int e = 3; e >= 0; --e) {
      const uint64_t q = mul_f32x2(x[e], y);
      uint64_t c = fma_f32x2(fma_f32x2(q, minus_s, x[e]), y, q);
      float c0, c1;
      if constexpr (kType == kFP16) {
        unpack_f32x2(c, c0, c1);
        c = pack_f32x2(fminf(fmaxf(c0, 0.f), 15.f), fminf(fmaxf(c1, 0.f), 15.f));
      }
      unpack_f32x2(add_f32x2(c, magic), c0, c1);
      w = (w * 16u + __float_as_uint(c1)) * 16u + __float_as_uint(c0);
    }
    w -= 0x4b400000u * 0x11111111u;
  } else {
    const float half = range > 0x1p100f ? 0.5f : 1.f;  // (exact for every value that counts next to such a range)
    sm = pack_bf16x2(__fdiv_rn(hi * half - lo * half, 15.f * half), lo);
    s = bf16_lo(sm);
#pragma unroll
    for (int e = 3; e >= 0; --e) {
      const float2 f = unpack_16x2<kType>((&raw.x)[e]);
      const float d[2] = {f.x * half - m * half, f.y * half - m * half};
#pragma unroll
      for (int i = 1; i >= 0; --i) {
        const float c = s != 0.f ? rintf(fminf(fmaxf(__fdiv_rn(d[i], s * half), 0.f), 15.f)) : 0.f;
        w = w * 16u + static_cast<uint32_t>(c);
      }
    }
  }
  *meta = sm;
  return w;
}

// Appends packed rows of K and V (bf16 or fp16): quantises each row, writes
// it at its sequence's next slot, its position, and a zero weight.
// HBM-bound: 4*D bytes read and D + D/8 + 8 written per row and head.
// 37281 tokens of 8 heads, D = 128: 46 us for 198 MB, 4.3 TB/s; the issue slots are
// busy three quarters of the time, so a division of its own for every value had
// taken 124 us and a search for the sequence in every head 74.
template <int D, int kType>
__global__ void __launch_bounds__(kC4RowsThreads, 4)
    attn_cache4_append_kernel(const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, Cache4Rows g, Cache4 c,
                              int heads, float* __restrict__ weight, int32_t* __restrict__ pos,
                              const int32_t* __restrict__ first_pos, int32_t* __restrict__ len_out) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x) % kC4RowLanes<D>;
  const int h0 = static_cast<int>(blockIdx.x) * heads, h1 = min(c.H, h0 + heads);
  for (int64_t row0 = static_cast<int64_t>(blockIdx.y) * kC4BlockRows<D>; row0 < g.rows;
       row0 += static_cast<int64_t>(gridDim.y) * kC4BlockRows<D>) {
    const int64_t row = row0 + threadIdx.x / kC4RowLanes<D>;
    const C4Row r = c4_row<true>(g, c, row);
    if (r.dropped && lane == 0 && h0 == 0) atomicOr(&g_attn_status, kC4Overflow);
    const int my_pos = r.at < 0 ? 0 : (first_pos != nullptr ? __ldg(first_pos + r.b) : max(__ldg(g.slot0 + r.b), 0)) + r.i;
    const int64_t from = r.at < 0 ? 0 : row;  // the others go through the motions: the statistics are whole warps'
    const uint16_t* kp = k + from * g.k_stride + h0 * D + lane * 8;
    const uint16_t* vp = v + from * g.v_stride + h0 * D + lane * 8;
    int64_t at = r.at + static_cast<int64_t>(h0) * c.cap;
    // the next head's values travel while this one's are quantised
    uint4 nk = __ldg(reinterpret_cast<const uint4*>(kp)), nv = __ldg(reinterpret_cast<const uint4*>(vp));
#pragma unroll 1
    for (int h = h0; h < h1; ++h, at += c.cap) {
      const uint4 xk = nk, xv = nv;
      if (h + 1 < h1) {
        kp += D;
        vp += D;
        nk = __ldg(reinterpret_cast<const uint4*>(kp));
        nv = __ldg(reinterpret_cast<const uint4*>(vp));
      }
      uint32_t mk, mv;
      const uint32_t wk = c4_quantise<kType>(xk, &mk), wv = c4_quantise<kType>(xv, &mv);
      if (r.at < 0) continue;
      reinterpret_cast<uint32_t*>(c.k)[at * (D / 8) + lane] = wk;
      reinterpret_cast<uint32_t*>(c.v)[at * (D / 8) + lane] = wv;
      if ((lane & 7) == 0) {
        c.km[at * (D / kC4Group) + (lane >> 3)] = mk;
        c.vm[at * (D / kC4Group) + (lane >> 3)] = mv;
      }
      if (lane == 0) {
        if (weight != nullptr) weight[at] = 0.f;
        if (pos != nullptr) pos[at] = my_pos;
      }
    }
  }
  if (len_out != nullptr && h0 == 0) {
    for (int64_t b = blockIdx.y * static_cast<int64_t>(blockDim.x) + threadIdx.x; b < g.B;
         b += static_cast<int64_t>(gridDim.y) * blockDim.x) {
      const int64_t l = static_cast<int64_t>(max(0, __ldg(g.slot0 + b))) + c4_rows_of(g, static_cast<int>(b));
      len_out[b] = static_cast<int32_t>(l < c.cap ? l : c.cap);
    }
  }
}

// The same update where len_out is the cache's own length: a launch behind
// the one whose blocks all read it.
__global__ void attn_cache4_grow_kernel(Cache4Rows g, int32_t* len, int cap) {
  grid_dependency_wait();
  grid_launch_dependents();
  for (int64_t b = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; b < g.B;
       b += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t l = static_cast<int64_t>(max(0, len[b])) + c4_rows_of(g, static_cast<int>(b));
    len[b] = static_cast<int32_t>(l < cap ? l : cap);
  }
}

// Reads entries back into packed rows: c*s + m, rounded once to the output's
// type.  c*s + m is exact in fp32 wherever s and m are within 2^12 of each
// other (4 + 8 bits of c*s against 8 of m).
// Codes become numbers by ORing them, where they are, into the mantissa of
// 2^23: 2^23 + c * 16^e, of which the sum with -2^23 is exact.
// 37281 rows of 8 heads, D = 128, to bf16: 35 us for 196 MB, 5.6 TB/s; with one
// head's codes in flight instead of two it took 37.
template <int D, int kType>
__global__ void __launch_bounds__(kC4RowsThreads)
    attn_cache4_read_kernel(void* __restrict__ k, void* __restrict__ v, Cache4Rows g, Cache4 c, int heads) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x) % kC4RowLanes<D>;
  const int h0 = static_cast<int>(blockIdx.x) * heads, h1 = min(c.H, h0 + heads);
  for (int64_t row0 = static_cast<int64_t>(blockIdx.y) * kC4BlockRows<D>; row0 < g.rows;
       row0 += static_cast<int64_t>(gridDim.y) * kC4BlockRows<D>) {
    const int64_t row = row0 + threadIdx.x / kC4RowLanes<D>;
    const C4Row r = c4_row<false>(g, c, row);
    if (r.at < 0) continue;
    int64_t at = r.at + static_cast<int64_t>(h0) * c.cap;
    // two heads' codes travel while this one's are turned into values
    uint32_t n[4], n2[4];
    const auto load = [&](uint32_t* n) {
      n[0] = __ldg(reinterpret_cast<const uint32_t*>(c.k) + at * (D / 8) + lane);
      n[1] = __ldg(reinterpret_cast<const uint32_t*>(c.v) + at * (D / 8) + lane);
      n[2] = __ldg(c.km + at * (D / kC4Group) + (lane >> 3));
      n[3] = __ldg(c.vm + at * (D / kC4Group) + (lane >> 3));
    };
    load(n);
    if (h0 + 1 < h1) {
      at += c.cap;
      load(n2);
    }
#pragma unroll 1
    for (int h = h0; h < h1; ++h) {
      const uint32_t wk = n[0], wv = n[1], mk = n[2], mv = n[3];
#pragma unroll
      for (int e = 0; e < 4; ++e) n[e] = n2[e];
      if (h + 2 < h1) {
        at += c.cap;
        load(n2);
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t w = kv ? wv : wk, sm = kv ? mv : mk, half[2] = {w, w >> 16};
        const float s = bf16_lo(sm), m = bf16_hi(sm);
        const uint64_t scale[2] = {pack_f32x2(s, s * 0x1p-4f), pack_f32x2(s * 0x1p-8f, s * 0x1p-12f)};
        const uint64_t minus = pack_f32x2(-8388608.f, -8388608.f), m2 = pack_f32x2(m, m);
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const uint32_t c0 = and_or(half[e >> 2], 15u << (4 * (e & 3)), 0x4b000000u);
          const uint32_t c1 = and_or(half[e >> 2], 15u << (4 * (e & 3) + 4), 0x4b000000u);
          unpack_f32x2(fma_f32x2(add_f32x2(pack_f32x2(__uint_as_float(c0), __uint_as_float(c1)), minus), scale[(e >> 1) & 1], m2),
                       x[e], x[e + 1]);
        }
        if (s < 0x1p-100f) {  // the scaled s may be subnormal
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = fmaf(static_cast<float>((w >> (4 * e)) & 15u), s, m);
        }
        const int64_t to = row * (kv ? g.v_stride : g.k_stride) + h * D + lane * 8;
        if constexpr (kType == kFP32) {
          float4* dst = reinterpret_cast<float4*>(static_cast<float*>(kv ? v : k) + to);
          dst[0] = make_float4(x[0], x[1], x[2], x[3]);
          dst[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(kv ? v : k) + to) =
              make_uint4(pack_16x2<kType>(x[0], x[1]), pack_16x2<kType>(x[2], x[3]), pack_16x2<kType>(x[4], x[5]),
                         pack_16x2<kType>(x[6], x[7]));
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Attention of one token per sequence over the cache
// ---------------------------------------------------------------------------
//
// For a group of G query heads that share a key head,
//     x_gj = scale * <q_g, k_j>,  O_g = sum_j softmax_j(x_g.) v_j.
// With k_j = s c + m in each group of 64 channels, the codes go through the
// tensor core, centred, and the scales are applied to sums:
//     <q, k_j>  = sum over groups of  s * <q, c - 8> + (m + 8 s) * sum q
//     sum_j p_j v_j = sum_j (p_j s) (c - 8) + sum_j p_j (m + 8 s).
// The products run in fp16 with fp32 sums, whatever the type of q and o:
//   * A code is ORed into the mantissa of 1024 (the conversion of 4-bit weights in
//     Y. J. Kim et al., "Who says elephants can't run", 2022): a low nibble gives
//     1024 + c, a high one, left where it is, 1024 + 16 c, and one fused
//     multiply-add turns either into a multiple of c - 8.  So two nibbles of a
//     16-bit half need one mask and one operation each, and one shift serves four
//     of the eight.
//   * Both are centred: a mean code of 7.5 would take bits from the sums.  And both
//     are normal numbers, K's (c - 8) * 2^-14: the tensor core lines its products up
//     by their exponents, and a subnormal's is that of the smallest normal number.
//     K's codes taken as they stand in the word, c * 2^-24 and c * 2^-20, need no
//     such operation (1 sequence of 131072 entries 36.5 us instead of 38.2, 64 of up
//     to 16000 with weights 131.1 instead of 133.0), but the logits then lost 3 to
//     4 bits against fp32 products; as it is they are as exact as those.
//   * q is scaled by a power of two that brings its head's largest channel to
//     2^4 .. 2^5, which fp16 holds to its 11 bits down to 2^-18 of it and to 2^-29
//     of it absolutely; the scale goes back into the logits.
//   * p s is held relative to a power of two T at or above every p s of that head
//     and group of channels when it was set, times 2^11: a tile that brings more
//     than 2^15 sets it anew, and O is rescaled, as it is when the running maximum
//     grows (p s of the keys so far shrinks with it, and so does T).  So p s has 11
//     bits down to 2^-25 of the largest and is off by 2^-36 T at most below.  It has
//     to be the largest product: relative to the largest s, one key of no weight
//     with an s 2^25 times the others' took the bits from all of them.
//
// mma.sync m16n8k16 serves here, with keys as the M rows of S^T = K Q^T, and
// channels as the M rows of O^T = V^T P^T: the A operands are then the cache's
// codes, turned into numbers in registers, and N = 8 is one block of up to 8
// query heads.  The pass is bound by HBM (4.5 bits a value) and by the
// instructions that unpack the codes, not by the products; tcgen05 would have the
// numbers written back to shared memory first.  The order of the channels within
// an MMA is free as long as both operands use the same one: slot (2i, 2i + 1)
// takes nibbles (e, e + 4) of a word, which one mask extracts together.
//
// Work split: the cache entries of all sequences and key heads, in tiles of 64
// keys, form one list, cut into equal contiguous shares, one per CTA, whatever
// the lengths are.  A CTA's share of one (sequence, key head) is a segment;
// its four warps take 16 keys of every tile each, with running statistics of
// their own, and join at the segment's end into one partial (m, l, O).  The
// merge kernel joins the partials of a row.  Where max_len is at most
// kC4DirectLen a CTA takes a whole row instead and writes O and LSE itself, and
// the weights where the row has all the heads of its key head: one launch, and
// without weights no workspace.  (One sequence of 701 entries, 16 heads, D = 64:
// 4.3 us on the GPU instead of 7.7, and 13 us on the host instead of 20.)

constexpr int kC4DecThreads = 128;  // 4 warps
constexpr int kC4TileKeys = 64;     // keys of a tile: 16 a warp
constexpr int kC4Heads = 8;         // query heads of a block (N of the MMA)
// Three CTAs an SM give a thread 168 registers, room for two tiles' chains of
// instructions side by side; with four (128, spills) it takes 145 us instead of
// 133 at 64 sequences of up to 16000 entries with weights, and 44.6 instead of
// 38.3 at one of 131072.  At D = 64, where a CTA takes a whole row, 128 registers
// do without spills, and four let more of the next call's rows start early (16
// sequences of 16 key heads, up to 1024 entries, with weights: 10.0 -> 7.9 us).
constexpr int kC4DecCtasPerSm = 3;
// Longest caches for which a CTA takes a whole row.  GPU time per call, that way
// against shares (us; lengths from half to all of the capacity; 1 sequence of 8 key
// heads, D = 128 | 64 of them | 16 of 16, D = 64):
//   1024           7.3 / 7.8   | 19.6 / 23.5 | 6.5 / 11.4
//   2048          10.7 / 8.0   | 34.7 / 34.9 | 10.5 / 14.4
//   4096          12.5 / 10.6  | 61.0 / 53.8 | 19.0 / 19.0
//   1024, weights  9.9 / 8.8   | 22.6 / 28.2 | 8.0 / 13.9
//   2048, weights 15.3 / 10.3  | 43.5 / 41.4 | 13.4 / 17.1
//   4096, weights 25.4 / 12.2  | 83.9 / 65.8 | 23.5 / 23.0
// On the GPU alone the border would lie lower for few rows, which leave most SMs
// idle (2048 entries of one sequence with weights: 5 us).  Shares take the host 4 us
// longer (a second launch, a workspace), and a call outside a graph waits for the
// host where the GPU needs less than 15: so 2048, whatever the rows.
constexpr int kC4DirectLen = 2048;
// Tiles' worth of time that a row costs a CTA.  1 sequence of 131072 | 32 of up to
// 4001 with weights | 64 of up to 16000 with weights: 38.3 | 29.9 | 132.8 us; with 3
// 37.4 | 31.6 | 137.0, with 12 38.4 | 31.9 | 134.1.
constexpr int kC4RowCost = 6;
// A GB300's SMs.  Workspaces are sized, and their use laid out, by this count,
// so that a size asked for on one device (or with none) holds on any.
constexpr int kC4WorkspaceSms = 152;

struct DecParams {
  Cache4 c;
  const uint16_t* q;  // [B][q_stride]: H_q rows of D
  int64_t q_stride;
  const int32_t* len;
  int B;
  int G;         // query heads per key head
  int HB;        // blocks of 8 of them
  int most;      // bound on the lengths
  float scale_log2;
  float* o_part;    // [slots][8][D], unnormalised
  float2* ml_part;  // [slots][8]: (m in log2 units, l)
  float* scores;    // [tile of a (sequence, key head)][G][64], units of kC4LogitUnit, or null
  uint16_t* o;      // [B][H*G][D]
  float* lse;       // [B][H*G]
  const float* w_in;
  float* w_out;     // [B][H][cap]
};

__device__ __forceinline__ int c4_tiles(const DecParams& p, int b) {
  return (c4_len(p.len, b, p.most) + kC4TileKeys - 1) / kC4TileKeys;
}

// The list that is cut into shares: each row (a sequence's key head, or block of
// query heads) that has entries counts `cost` units, for its start and its end,
// and one for each of its tiles.  (Without the fixed part, a CTA whose share held
// eight one-token rows took three times as long as the others.)
//
// Before a sequence lie so many tiles and so many sequences with entries, per
// row; both in one 64-bit number.
constexpr int64_t kC4Tiles = (1ll << 40) - 1;
__device__ __forceinline__ int64_t c4_count(int nt) { return nt + (nt > 0 ? 1ll << 40 : 0ll); }
__device__ __forceinline__ int64_t c4_units(int64_t count, int cost) { return (count & kC4Tiles) + cost * (count >> 40); }
__device__ __forceinline__ int c4_row_units(int nt, int cost) { return nt > 0 ? nt + cost : 0; }

// Counts over all sequences, over those before this thread's stripe of them and
// over its stripe.  All threads of the block call it.
__device__ __forceinline__ int64_t c4_total(const DecParams& p, int64_t* warp_sums, int64_t* mine_before, int64_t* mine) {
  const int tid = static_cast<int>(threadIdx.x), n_thr = static_cast<int>(blockDim.x);
  const int stripe = (p.B + n_thr - 1) / n_thr;
  const int b0 = min(p.B, tid * stripe), b1 = min(p.B, b0 + stripe);
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += c4_count(c4_tiles(p, b));
  int64_t incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, off);
    if ((tid & 31) >= off) incl += y;
  }
  if ((tid & 31) == 31) warp_sums[tid >> 5] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < n_thr / 32; ++w) {
    if (w < (tid >> 5)) before += warp_sums[w];
    total += warp_sums[w];
  }
  *mine_before = before + incl - sum;
  *mine = sum;
  return total;
}
// The sequence with unit y (of one row's units; 0 <= y < their sum) and the
// counts before it: the thread whose stripe holds it walks the stripe and
// tells the block.
__device__ __forceinline__ void c4_find(const DecParams& p, int64_t y, int cost, int64_t mine_before, int64_t mine,
                                        int* b_out, int64_t* before_out) {
  if (c4_units(mine_before, cost) <= y && y < c4_units(mine_before + mine, cost)) {
    const int stripe = (p.B + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    int b = static_cast<int>(threadIdx.x) * stripe;
    int64_t at = mine_before;
    while (true) {
      const int64_t next = at + c4_count(c4_tiles(p, b));
      if (y < c4_units(next, cost)) break;
      at = next;
      ++b;
    }
    *b_out = b;
    *before_out = at;
  }
}

// A block's walk over its share [x, end) of a list with `rows` rows a sequence.
struct C4Walk {
  int64_t x, end;
  int64_t before;   // counts before sequence b
  int b, n, nt;     // sequence, its entries and tiles
  int row, t0, t1;  // row of the sequence, tiles of it
  // Moves to the next row whose tiles the share holds; false at the share's end.
  __device__ bool next(const DecParams& p, int rows, int cost) {
    while (x < end) {
      n = c4_len(p.len, b, p.most);
      nt = (n + kC4TileKeys - 1) / kC4TileKeys;
      const int units = c4_row_units(nt, cost);
      const int64_t at = x - c4_units(before, cost) * rows;
      if (at >= static_cast<int64_t>(units) * rows) {
        before += c4_count(nt);
        ++b;
        continue;
      }
      row = static_cast<int>(at / units);
      const int u0 = static_cast<int>(at - static_cast<int64_t>(row) * units);
      const int u1 = static_cast<int>(end - x < units - u0 ? u0 + (end - x) : units);
      x += u1 - u0;
      t0 = max(0, u0 - cost);
      t1 = u1 - cost;
      if (t0 < t1) return true;
    }
    return false;
  }
};

__device__ __forceinline__ void mma_16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same onto zero.
__device__ __forceinline__ void mma_16816_zero(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Codes as fp16 numbers.  K's: (c - 8) * 2^-14 of the low nibbles of both 16-bit
// halves' low bytes, and of the high nibbles: exact, and normal numbers.
__device__ __forceinline__ uint32_t c4_key_low(uint32_t w) {  // (1024 + c) 2^-14 - 1032 * 2^-14
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(and_or(w, 0x000f000fu, 0x64006400u)), "r"(0x04000400u), "r"(0xac08ac08u));
  return r;
}
__device__ __forceinline__ uint32_t c4_key_high(uint32_t w) {  // (1024 + 16 c) 2^-18 - 72 * 2^-14
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(and_or(w, 0x00f000f0u, 0x64006400u)), "r"(0x00400040u), "r"(0x9c809c80u));
  return r;
}
// V's: c - 8 of the same nibbles: exact.
__device__ __forceinline__ uint32_t c4_low(uint32_t w) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(and_or(w, 0x000f000fu, 0x64006400u)), "r"(0x64086408u));
  return r;
}
__device__ __forceinline__ uint32_t c4_high(uint32_t w) {  // (1024 + 16 c) / 16 - 72
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(and_or(w, 0x00f000f0u, 0x64006400u)), "r"(0x2c002c00u), "r"(0xd480d480u));
  return r;
}

// 8 x 8 matrix of 16-bit values across the warp, transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A warp's 16 keys of a tile travel through a ring of shared-memory stages of
// its own, filled by asynchronous copies: four stages, and 12 warps an SM, are up
// to 110 KB in flight.  Loads into registers kept some 40 KB there and took a fifth
// longer (64 sequences of up to 16000 entries, one tile a step).
// A stage is K codes, V codes, K meta, V meta, row by row.  The 16-byte pieces of
// a row are swapped so that eight rows' pieces of one number, which ldmatrix reads
// at once, lie in different banks: a row has 4 pieces (D = 128) or 2, and 8 fill
// the 32 banks.
template <int D>
struct C4Ring {
  static constexpr int kStages = 4;
  static constexpr int kRow = D / 2;             // bytes of codes a row
  static constexpr int kMeta = D / kC4Group * 4;  // bytes of (s, m) a row
  static constexpr int kV = 16 * kRow;
  static constexpr int kKm = 32 * kRow;
  static constexpr int kVm = kKm + 16 * kMeta;
  static constexpr int kStage = kVm + 16 * kMeta;
  static constexpr int kWarp = kStages * kStage;
  // byte of row `row`'s piece; 8 rows further its place is the same
  __device__ static uint32_t at(int row, int piece) {
    return static_cast<uint32_t>(row * kRow + (piece ^ (D == 128 ? (row >> 1) & 3 : (row >> 2) & 1)) * 16);
  }
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int kBytes>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// What this lane copies of every tile: 16-byte pieces of K and V codes and one
// row's meta (lanes 0-15 of K, 16-31 of V).  The pointers are the next tile's.
template <int D>
struct C4Copy {
  using R = C4Ring<D>;
  static constexpr int kPieces = D / 64;  // of K, and of V: the second one is 8 rows further
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* meta;
  uint32_t dst, meta_dst;
  int row, meta_row;
  __device__ void start(const Cache4& c, int64_t key0, int lane, uint32_t ring) {
    constexpr int kPerRow = R::kRow / 16;
    row = lane / kPerRow;
    meta_row = lane & 15;
    const int piece = lane % kPerRow;
    k = c.k + (key0 + row) * R::kRow + piece * 16;
    v = c.v + (key0 + row) * R::kRow + piece * 16;
    meta = reinterpret_cast<const uint8_t*>(lane < 16 ? c.km : c.vm) + (key0 + meta_row) * R::kMeta;
    dst = ring + R::at(row, piece);
    meta_dst = ring + R::kKm + static_cast<uint32_t>(lane) * R::kMeta;
  }
  __device__ void issue(uint32_t stage) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      cp_async_16(dst + stage + i * 8 * R::kRow, k + i * 8 * R::kRow);
      cp_async_16(dst + stage + R::kV + i * 8 * R::kRow, v + i * 8 * R::kRow);
    }
    cp_async_small<R::kMeta>(meta_dst + stage, meta);
    k += kC4TileKeys * R::kRow;
    v += kC4TileKeys * R::kRow;
    meta += kC4TileKeys * R::kMeta;
  }
  // The last tile, of which `left` < 16 keys exist: rows past the end take the
  // last one again.  They are masked, and nothing is read that was never written.
  __device__ void issue_tail(uint32_t stage, int left) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int off = (min(row + 8 * i, left - 1) - row) * R::kRow;
      cp_async_16(dst + stage + i * 8 * R::kRow, k + off);
      cp_async_16(dst + stage + R::kV + i * 8 * R::kRow, v + off);
    }
    cp_async_small<R::kMeta>(meta_dst + stage, meta + (min(meta_row, left - 1) - meta_row) * R::kMeta);
  }
};

// This lane's shared-memory addresses in stage 0: the piece that it names to
// ldmatrix (matrices 0 and 2: rows 0-7, 1 and 3: rows 8-15; 0 and 1: a group's
// first 32 channels, 2 and 3: the others), and its (s, m).
template <int D>
struct C4Lane {
  uint32_t codes[D / kC4Group], meta;
  __device__ void start(uint32_t ring, int lane) {
    using R = C4Ring<D>;
#pragma unroll
    for (int g = 0; g < D / kC4Group; ++g) codes[g] = ring + R::at(lane & 15, 2 * g + (lane >> 4));
    meta = ring + R::kKm + static_cast<uint32_t>((lane >> 2) * R::kMeta);
  }
};
__device__ __forceinline__ void ldmatrix_x4(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_b32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
// The (s, m) of keys r and r + 8, of K or (at kVm - kKm) of V.
template <int D>
__device__ __forceinline__ void c4_load_meta(uint32_t (*sm)[D / kC4Group], uint32_t at) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (D == 128) {
      const uint2 a = ld_shared_v2(at + i * 8 * C4Ring<D>::kMeta);
      sm[i][0] = a.x, sm[i][1] = a.y;
    } else {
      sm[i][0] = ld_shared_b32(at + i * 8 * C4Ring<D>::kMeta);
    }
  }
}

// A tile's logits, and what is compared with them, are log2 units over this: so
// they come out of the MMAs, and the multiplication joins the subtraction in the
// exponent.
constexpr float kC4LogitUnit = 1024.f;

// Q of a block of up to 8 heads as B operands, and what goes with it.
template <int D>
struct C4Query {
  static constexpr int kGroups = D / kC4Group;
  uint32_t q[kGroups][4][2];  // head r, in the channel order of the K words
  float sum[kGroups][2];      // of heads 2c, 2c + 1, over a group's channels, in the units of the MMAs' sums
  float scale[2];             // logits of heads 2c, 2c + 1, in units of kC4LogitUnit
};
template <int D, int kType>
__device__ __forceinline__ void c4_load_query(C4Query<D>& t, const uint16_t* rows, int heads, float scale_log2, int r, int c) {
  constexpr int kG = D / kC4Group;
  const bool there = r < heads;
  const uint16_t* qr = rows + (there ? r : 0) * D;
  uint32_t raw[kG][8];
#pragma unroll
  for (int g = 0; g < kG; ++g)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (there) x = __ldg(reinterpret_cast<const uint4*>(qr + g * kC4Group + w * 32 + c * 8));
      raw[g][4 * w] = x.x, raw[g][4 * w + 1] = x.y, raw[g][4 * w + 2] = x.z, raw[g][4 * w + 3] = x.w;
    }
  // A head's q in fp16, times 2^4 / 2^E for its largest in [2^E, 2^(E+1)).
  float top = 0.f;
#pragma unroll
  for (int g = 0; g < kG; ++g)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = unpack_16x2<kType>(raw[g][i]);
      top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
    }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // 2^-E within 2^-126 .. 2^100; 1 for 0, and for infinity, which stays one
  const int e = static_cast<int>(__float_as_uint(top) >> 23);
  const int f = top == 0.f || e == 255 ? 127 : min(max(254 - e, 1), 227);
  const float fwd = __uint_as_float(static_cast<uint32_t>(f + 4) << 23);
  const float back = __uint_as_float(static_cast<uint32_t>(254 - f) << 23);
#pragma unroll
  for (int g = 0; g < kG; ++g)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = unpack_16x2<kType>(raw[g][i]);
      raw[g][i] = pack_f16x2(x.x * fwd, x.y * fwd);
    }
  t.scale[0] = scale_log2 * __shfl_sync(0xffffffffu, back, 8 * c);
  t.scale[1] = scale_log2 * __shfl_sync(0xffffffffu, back, 8 * c + 4);
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = unpack_f16x2(raw[g][i]);
      sum += f.x + f.y;
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    sum *= 0x1p-14f;  // the MMAs' sums: 2^4 q times (c - 8) * 2^-14
    t.sum[g][0] = __shfl_sync(0xffffffffu, sum, 8 * c);
    t.sum[g][1] = __shfl_sync(0xffffffffu, sum, 8 * c + 4);
    // nibbles e and e + 4 of a word meet in one register: channels (0, 4),
    // (1, 5) go into one MMA, (2, 6), (3, 7) into the next
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint32_t* e = raw[g] + 4 * w;
      t.q[g][2 * w][0] = __byte_perm(e[0], e[2], 0x5410);
      t.q[g][2 * w][1] = __byte_perm(e[0], e[2], 0x7632);
      t.q[g][2 * w + 1][0] = __byte_perm(e[1], e[3], 0x5410);
      t.q[g][2 * w + 1][1] = __byte_perm(e[1], e[3], 0x7632);
    }
  }
}

// Running state of a warp: heads 2c and 2c + 1.
template <int D>
struct C4State {
  static constexpr int kGroups = D / kC4Group;
  float ref[2];              // what p is relative to, units of kC4LogitUnit
  float sub[2];              // the same in log2 units, 0 instead of -inf
  float most[2];             // 8 log2 units above ref
  float l[2];                // this lane's share of sum p
  float bias[kGroups][2];    // this lane's share of sum p (m + 8 s)
  float inv[kGroups][2];     // what p s is held times, a power of two (0 at first)
  float o[kGroups][4][4];    // O^T, times inv: channels 64g + 4r + u (+ 32), heads 2c, 2c + 1
};
// 1 / inv, 0 where inv is.
__device__ __forceinline__ float c4_unit(float inv) {
  return inv == 0.f ? 0.f : __uint_as_float((254u << 23) - __float_as_uint(inv));
}

// Logits of a tile's 16 keys: keys r, r, r + 8, r + 8 and heads 2c, 2c + 1, 2c,
// 2c + 1.  ldmatrix gives this lane word c (8 channels) of a piece of rows r and
// r + 8.
template <int D>
__device__ __forceinline__ void c4_scores(float* xs, const C4Lane<D>& p, uint32_t stage, const C4Query<D>& q) {
  using R = C4Ring<D>;
  constexpr int kG = D / kC4Group;
  uint32_t sm[2][kG];
  c4_load_meta<D>(sm, p.meta + stage);
#pragma unroll
  for (int e = 0; e < 4; ++e) xs[e] = 0.f;
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    uint32_t w[4];
    ldmatrix_x4(w, p.codes[g] + stage);
    float d[4];
    mma_16816_zero(d, c4_key_low(w[0]), c4_key_low(w[1]), c4_key_high(w[0]), c4_key_high(w[1]), q.q[g][0][0], q.q[g][0][1]);
    mma_16816(d, c4_key_low(w[0] >> 8), c4_key_low(w[1] >> 8), c4_key_high(w[0] >> 8), c4_key_high(w[1] >> 8), q.q[g][1][0],
              q.q[g][1][1]);
    mma_16816(d, c4_key_low(w[2]), c4_key_low(w[3]), c4_key_high(w[2]), c4_key_high(w[3]), q.q[g][2][0], q.q[g][2][1]);
    mma_16816(d, c4_key_low(w[2] >> 8), c4_key_low(w[3] >> 8), c4_key_high(w[2] >> 8), c4_key_high(w[3] >> 8), q.q[g][3][0],
              q.q[g][3][1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float s = bf16_lo(sm[i][g]), m = fmaf(8.f, s, bf16_hi(sm[i][g]));
      xs[2 * i] = fmaf(s, d[2 * i], fmaf(m, q.sum[g][0], xs[2 * i]));
      xs[2 * i + 1] = fmaf(s, d[2 * i + 1], fmaf(m, q.sum[g][1], xs[2 * i + 1]));
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) xs[e] *= q.scale[e & 1];
}

// p of a tile's 16 keys and, in fp16, p s times st.inv; pr as c4_scores lays out the
// logits.  Returns the largest of the products and `most`.
template <int D>
__device__ __forceinline__ float c4_weigh(float* pr, uint32_t (*ps)[2], const float* xs, const C4State<D>& st,
                                          const uint32_t (*sm)[D / kC4Group], float most) {
#pragma unroll
  for (int e = 0; e < 4; ++e) pr[e] = ex2_approx(fmaf(xs[e], kC4LogitUnit, -st.sub[e & 1]));
#pragma unroll
  for (int g = 0; g < D / kC4Group; ++g)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // (s last: a p of 0 stays 0, whatever s times inv is)
      const float s = bf16_lo(sm[i][g]), y0 = pr[2 * i] * st.inv[g][0] * s, y1 = pr[2 * i + 1] * st.inv[g][1] * s;
      most = max3f(most, fabsf(y0), fabsf(y1));
      ps[g][i] = pack_f16x2(y0, y1);
    }
  return most;
}

// O^T += V^T P^T over a tile's 16 keys; pr and ps as c4_weigh leaves them.
// ldmatrix transposes units of 16 bits, 4 channels: this lane gets unit r of a
// piece from keys 2c and 2c + 1 side by side (and from 2c + 8, 2c + 9).
template <int D>
__device__ __forceinline__ void c4_values(C4State<D>& st, const float* pr, const uint32_t (*ps)[2],
                                          const uint32_t (*sm)[D / kC4Group], const C4Lane<D>& p, uint32_t stage) {
#pragma unroll
  for (int g = 0; g < D / kC4Group; ++g) {
    uint32_t pb[2];  // P^T as the B operand: keys 0-7 and 8-15
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float mm = fmaf(8.f, bf16_lo(sm[i][g]), bf16_hi(sm[i][g]));
      st.bias[g][0] = fmaf(pr[2 * i], mm, st.bias[g][0]);
      st.bias[g][1] = fmaf(pr[2 * i + 1], mm, st.bias[g][1]);
      pb[i] = movmatrix_trans(ps[g][i]);
    }
    uint32_t w[4];
    ldmatrix_x4_trans(w, p.codes[g] + stage + C4Ring<D>::kV);
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // rows r: channels 4r + 2j (+ 1); rows r + 8: those + 32
      const uint32_t a0 = w[0] >> (8 * j), a1 = w[2] >> (8 * j), a2 = w[1] >> (8 * j), a3 = w[3] >> (8 * j);
      mma_16816(st.o[g][2 * j], c4_low(a0), c4_low(a1), c4_low(a2), c4_low(a3), pb[0], pb[1]);
      mma_16816(st.o[g][2 * j + 1], c4_high(a0), c4_high(a1), c4_high(a2), c4_high(a3), pb[0], pb[1]);
    }
  }
}

// kN tiles' 16 keys each, in stages stage[0], ...; with kTail the first `left`
// keys of the (one) tile exist.  `scores`: where head 2c's score of key
// r of the first tile goes, [tile][head][64 keys], tiles sc_step apart.
template <int D, bool kWeight, bool kTail, int kN>
__device__ __forceinline__ void c4_step(C4State<D>& st, const C4Lane<D>& p, const uint32_t* stage, const C4Query<D>& q,
                                        int r, int left, float* scores, int64_t sc_step, bool head0, bool head1) {
  using R = C4Ring<D>;
  constexpr int kG = D / kC4Group;
  float xs[kN][4];
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    c4_scores<D>(xs[n], p, stage[n], q);
    if constexpr (kTail) {
      if (r >= left) xs[n][0] = xs[n][1] = -INFINITY;
      if (r + 8 >= left) xs[n][2] = xs[n][3] = -INFINITY;
    }
    if constexpr (kWeight) {
      float* dst = scores + n * sc_step;
      if (head0) {
        dst[0] = xs[n][0];
        dst[8] = xs[n][2];
      }
      if (head1) {
        dst[kC4TileKeys] = xs[n][1];
        dst[kC4TileKeys + 8] = xs[n][3];
      }
    }
  }
  uint32_t sm[kN][2][kG], ps[kN][kG][2];
  float pr[kN][4], top[2] = {-INFINITY, -INFINITY}, most = 0.f;
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    c4_load_meta<D>(sm[n], p.meta + stage[n] + (R::kVm - R::kKm));
#pragma unroll
    for (int e = 0; e < 2; ++e) top[e] = max3f(top[e], xs[n][e], xs[n][2 + e]);
    most = c4_weigh<D>(pr[n], ps[n], xs[n], st, sm[n], most);
  }
  // New references only where a score exceeds the old one by 2^8 or a product fp16's
  // range: p stays below 2^8, and most tiles need one vote instead of reductions and
  // a rescale.  (Where all scores are NaN there is no reference, and none is needed.)
  if (__any_sync(0xffffffffu, (top[0] > st.most[0]) | (top[1] > st.most[1]) | (most > 0x1p15f))) {
    float a[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], off));
      // a reference that has held moves only when it has to: p of the keys so
      // far keeps its bits
      const float to = top[e] > st.most[e] ? top[e] : st.ref[e];
      a[e] = to == st.ref[e] ? 1.f : ex2_approx((st.ref[e] - to) * kC4LogitUnit);
      st.ref[e] = to;
      st.sub[e] = to == -INFINITY ? 0.f : to * kC4LogitUnit;
      st.most[e] = to + kRescaleLog2 / kC4LogitUnit;
      st.l[e] *= a[e];
    }
    // T / 2^16 of a head and group (p s itself may be beyond fp32's range): the next
    // power of two above these tiles' products, or the old one as far as it has not
    // shrunk with p
#pragma unroll
    for (int g = 0; g < kG; ++g)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = 0.f;
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            x = fmaxf(x, fabsf(ex2_approx(fmaf(xs[n][2 * i + e], kC4LogitUnit, -st.sub[e])) * (bf16_lo(sm[n][i][g]) * 0x1p-16f)));
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
        const float old = c4_unit(st.inv[g][e]) * 0x1p-5f * a[e];
        const uint32_t up = max((__float_as_uint(x) + 0x007fffffu) & 0x7f800000u, __float_as_uint(old) & 0x7f800000u);
        const uint32_t to = min(max(up, 1u << 23), 247u << 23);  // inv within 2^-125 .. 2^121
        const float f = old * __uint_as_float((254u << 23) - to);
        st.inv[g][e] = __uint_as_float((249u << 23) - to);  // 2^-5 / to: 2^11 / T
        st.bias[g][e] *= a[e];
#pragma unroll
        for (int u = 0; u < 4; ++u) st.o[g][u][e] *= f, st.o[g][u][2 + e] *= f;
      }
#pragma unroll
    for (int n = 0; n < kN; ++n) c4_weigh<D>(pr[n], ps[n], xs[n], st, sm[n], 0.f);
  }
#pragma unroll
  for (int n = 0; n < kN; ++n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) st.l[e & 1] += pr[n][e];
    c4_values<D>(st, pr[n], ps[n], sm[n], p, stage[n]);
  }
}

// Adds the weights of tiles t0 .. t1 - 1 of a (sequence, key head) with n
// entries: exp2(logit - lse) summed over the heads of its group.  16 threads a
// tile, 4 keys each.  `scores`: of the row's tile 0, [tile][G][64]; kOwn: written
// by this block before a barrier, else by an earlier kernel.
template <bool kOwn>
__device__ __forceinline__ void c4_add_weights(const DecParams& p, int b, int h, int n, int t0, int t1, const float* scores,
                                               const float* lse_s) {
  const int k0 = (static_cast<int>(threadIdx.x) & 15) * 4;
  for (int t = t0 + (static_cast<int>(threadIdx.x) >> 4); t < t1; t += static_cast<int>(blockDim.x) >> 4) {
    const int64_t at = (static_cast<int64_t>(b) * p.c.H + h) * p.c.cap + static_cast<int64_t>(t) * kC4TileKeys + k0;
    const int left = n - t * kC4TileKeys - k0;  // of these 4 keys on
    const float4* src = reinterpret_cast<const float4*>(scores + static_cast<int64_t>(t) * p.G * kC4TileKeys + k0);
    float sum[4] = {0.f, 0.f, 0.f, 0.f}, in[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) in[e] = e < left ? p.w_in[at + e] : 0.f;
#pragma unroll 8
    for (int g = 0; g < p.G; ++g) {
      const float4 x = kOwn ? src[g * (kC4TileKeys / 4)] : __ldg(src + g * (kC4TileKeys / 4));
      const float z = lse_s[g];
      sum[0] += ex2_approx(fmaf(x.x, kC4LogitUnit, -z));
      sum[1] += ex2_approx(fmaf(x.y, kC4LogitUnit, -z));
      sum[2] += ex2_approx(fmaf(x.z, kC4LogitUnit, -z));
      sum[3] += ex2_approx(fmaf(x.w, kC4LogitUnit, -z));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) p.w_out[at + e] = in[e] + sum[e];
  }
}

// kDirect: CTA x takes the whole of row x (with weights: one block of heads a
// key head, so the row has all of an entry's weight).
template <int D, int kType, bool kWeight, bool kDirect>
__global__ void __launch_bounds__(kC4DecThreads, D == 64 && kDirect ? 4 : kC4DecCtasPerSm)
    attn_cache4_decode_kernel(const DecParams p) {
  constexpr int kG = D / kC4Group;
  constexpr int kWarps = kC4DecThreads / 32;
  using Ring = C4Ring<D>;
  __shared__ __align__(128) uint8_t ring_s[kWarps * Ring::kWarp];
  // the warps' O at a segment's end, when the ring is empty
  float(*const o_s)[kC4Heads][D + 4] = reinterpret_cast<float(*)[kC4Heads][D + 4]>(ring_s);
  static_assert(sizeof(float) * kWarps * kC4Heads * (D + 4) <= sizeof(ring_s), "O in the ring");
  __shared__ float2 ml_s[kWarps][kC4Heads];
  __shared__ float lse_s[kC4Heads];
  __shared__ int64_t sums_s[kWarps];
  __shared__ int64_t before_s;
  __shared__ int b_s;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  grid_dependency_wait();
  grid_launch_dependents();  // the merge kernel's blocks come as this one's leave
  const int rows_per_b = p.c.H * p.HB;
  C4Walk w;
  if constexpr (kDirect) {
    w.b = static_cast<int>(blockIdx.x) / rows_per_b;
    w.row = static_cast<int>(blockIdx.x) % rows_per_b;
    w.n = c4_len(p.len, w.b, p.most);
    w.t0 = 0;
    w.t1 = (w.n + kC4TileKeys - 1) / kC4TileKeys;
  } else {
    int64_t mine_before, mine;
    const int64_t total = c4_units(c4_total(p, sums_s, &mine_before, &mine), kC4RowCost) * rows_per_b;
    const int64_t share = (total + gridDim.x - 1) / gridDim.x;
    w.x = static_cast<int64_t>(blockIdx.x) * share;
    w.end = w.x + share < total ? w.x + share : total;
    if (w.x >= w.end) return;
    c4_find(p, w.x / rows_per_b, kC4RowCost, mine_before, mine, &b_s, &before_s);
    __syncthreads();
    w.b = b_s;
    w.before = before_s;
  }
  const uint32_t ring = smem_u32(ring_s) + static_cast<uint32_t>(warp * Ring::kWarp);
  C4Lane<D> at;
  at.start(ring, lane);
  for (bool once = true; kDirect ? once : w.next(p, rows_per_b, kC4RowCost); once = false) {
    const int b = w.b, n = w.n, in_b = w.row, t0 = w.t0, t1 = w.t1;
    const int h = in_b / p.HB, hb = in_b % p.HB;
    const int heads = min(kC4Heads, p.G - hb * kC4Heads);

    const int64_t row_base = (static_cast<int64_t>(b) * p.c.H + h) * p.c.cap;
    // This warp's keys of its tiles: 16 of each of `full`, then `last` < 16.
    const int64_t there = n - (static_cast<int64_t>(t0) * kC4TileKeys + warp * 16);  // keys from its first on
    const int full = there < 16 ? 0 : static_cast<int>(min(static_cast<int64_t>(t1 - t0), (there - 16) / kC4TileKeys + 1));
    const int last = full < t1 - t0 ? static_cast<int>(max(static_cast<int64_t>(0), there - static_cast<int64_t>(full) * kC4TileKeys)) : 0;
    C4Copy<D> copy;
    copy.start(p.c, row_base + static_cast<int64_t>(t0) * kC4TileKeys + warp * 16, lane, ring);
    const auto fetch = [&](int i, uint32_t stage) {
      if (i < full)
        copy.issue(stage);
      else if (i == full && last > 0)
        copy.issue_tail(stage, last);
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < Ring::kStages - 1; ++i) fetch(i, static_cast<uint32_t>(i * Ring::kStage));
    C4Query<D> q;
    c4_load_query<D, kType>(q, p.q + b * p.q_stride + static_cast<int64_t>(h * p.G + hb * kC4Heads) * D, heads, p.scale_log2,
                            r, c);
    C4State<D> st;
#pragma unroll
    for (int e = 0; e < 2; ++e) st.ref[e] = st.most[e] = -INFINITY, st.sub[e] = st.l[e] = 0.f;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      st.inv[g][0] = st.inv[g][1] = st.bias[g][0] = st.bias[g][1] = 0.f;
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[g][u][e] = 0.f;
    }
    // scores of (sequence, key head): its tiles in list order without the head blocks
    float* sc = kWeight ? p.scores + ((kDirect ? (static_cast<int64_t>(b) * p.c.H + h) * ((p.most + kC4TileKeys - 1) / kC4TileKeys)
                                           : (w.before & kC4Tiles) * p.c.H + static_cast<int64_t>(h) * w.nt + t0) * p.G + hb * kC4Heads + 2 * c) * kC4TileKeys +
                              warp * 16 + r
                        : nullptr;
    const int64_t sc_step = static_cast<int64_t>(p.G) * kC4TileKeys;
    const bool head0 = 2 * c < heads, head1 = 2 * c + 1 < heads;
    // Two tiles at a time (one vote, and two chains of instructions to overlap),
    // then the odd one, then the one that ends inside.
    int i = 0;
    uint32_t pair = 0u;  // stage of tile i; of i + 1: the next
    for (; i + 2 <= full; i += 2) {
      cp_async_wait<Ring::kStages - 3>();  // this lane's copies of tiles i and i + 1, ...
      __syncwarp();                        // ... and every lane's; the stage before is consumed
      const uint32_t stage[2] = {pair, pair + Ring::kStage};
      fetch(i + Ring::kStages - 1, (pair == 0u ? Ring::kStages * Ring::kStage : pair) - Ring::kStage);
      c4_step<D, kWeight, false, 2>(st, at, stage, q, r, 16, sc, sc_step, head0, head1);
      __syncwarp();
      fetch(i + Ring::kStages, pair);
      pair = pair == (Ring::kStages - 2) * Ring::kStage ? 0u : pair + 2 * Ring::kStage;
      if (kWeight) sc += 2 * sc_step;
    }
    if (i < full) {
      cp_async_wait<Ring::kStages - 3>();
      __syncwarp();
      const uint32_t stage[1] = {pair};
      c4_step<D, kWeight, false, 1>(st, at, stage, q, r, 16, sc, sc_step, head0, head1);
      if (kWeight) sc += sc_step;
      pair += Ring::kStage;
      ++i;
    }
    if (last > 0) {
      cp_async_wait<0>();
      __syncwarp();
      const uint32_t stage[1] = {pair};
      c4_step<D, kWeight, true, 1>(st, at, stage, q, r, last, sc, sc_step, head0, head1);
    }
    __syncthreads();  // the ring is empty (the copies of every tile were waited for) and read

    // Join the four warps: statistics over the lanes of a head, then O
    // relative to the segment's own maximum.
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        st.l[e] += __shfl_xor_sync(0xffffffffu, st.l[e], off);
#pragma unroll
        for (int g = 0; g < kG; ++g) st.bias[g][e] += __shfl_xor_sync(0xffffffffu, st.bias[g][e], off);
      }
    }
#pragma unroll
    for (int g = 0; g < kG; ++g)
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o_s[warp][2 * c + (e & 1)][g * kC4Group + 4 * r + u + 32 * (e >> 1)] =
              fmaf(st.o[g][u][e], c4_unit(st.inv[g][e & 1]), st.bias[g][e & 1]);
    if (r == 0) {
      ml_s[warp][2 * c] = make_float2(st.ref[0] * kC4LogitUnit, st.l[0]);
      ml_s[warp][2 * c + 1] = make_float2(st.ref[1] * kC4LogitUnit, st.l[1]);
    }
    __syncthreads();
    if constexpr (kDirect) {
      for (int i = tid; i < heads * D / 2; i += kC4DecThreads) {
        const int hd = i / (D / 2), d = i % (D / 2) * 2;
        float top = -INFINITY, x0 = 0.f, x1 = 0.f, ls = 0.f;
#pragma unroll
        for (int i2 = 0; i2 < kWarps; ++i2) top = fmaxf(top, ml_s[i2][hd].x);
#pragma unroll
        for (int i2 = 0; i2 < kWarps; ++i2) {
          const float a = top == -INFINITY ? 0.f : ex2_approx(ml_s[i2][hd].x - top);
          x0 = fmaf(a, o_s[i2][hd][d], x0);
          x1 = fmaf(a, o_s[i2][hd][d + 1], x1);
          ls = fmaf(a, ml_s[i2][hd].y, ls);
        }
        const float inv = ls == 0.f ? 0.f : 1.f / ls;  // 0: no entries
        const int64_t row = (static_cast<int64_t>(b) * p.c.H + h) * p.G + hb * kC4Heads + hd;
        *reinterpret_cast<uint32_t*>(p.o + row * D + d) = pack_16x2<kType>(x0 * inv, x1 * inv);
        if (d == 0) {
          p.lse[row] = ls == 0.f ? -INFINITY : (top + log2f(ls)) * kLn2;
          if (kWeight) lse_s[hd] = top + log2f(ls);
        }
      }
      if constexpr (kWeight) {
        __syncthreads();
        c4_add_weights<true>(p, b, h, n, t0, t1,
                             p.scores + (static_cast<int64_t>(b) * p.c.H + h) * ((p.most + kC4TileKeys - 1) / kC4TileKeys) * p.G * kC4TileKeys,
                             lse_s);
      }
    } else {
      const int64_t slot = blockIdx.x + static_cast<int64_t>(b) * rows_per_b + in_b;
      for (int i = tid; i < heads * D; i += kC4DecThreads) {
        const int hd = i / D, d = i % D;
        float top = -INFINITY;
#pragma unroll
        for (int i2 = 0; i2 < kWarps; ++i2) top = fmaxf(top, ml_s[i2][hd].x);
        float sum = 0.f, ls = 0.f;
#pragma unroll
        for (int i2 = 0; i2 < kWarps; ++i2) {
          const float a = top == -INFINITY ? 0.f : ex2_approx(ml_s[i2][hd].x - top);
          sum = fmaf(a, o_s[i2][hd][d], sum);
          ls = fmaf(a, ml_s[i2][hd].y, ls);
        }
        p.o_part[(slot * kC4Heads + hd) * D + d] = sum;
        if (d == 0) p.ml_part[slot * kC4Heads + hd] = make_float2(top, ls);
      }
      __syncthreads();
    }
  }
}

struct DecMergeParams {
  DecParams d;
  int dec_grid;  // CTAs of the decode kernel: the shares
  int warps;     // of the merge kernel that share a row's partials
  unsigned weight_blocks;  // blocks that add weights; those behind them join rows
};

constexpr int kC4MergeThreads = 256;
constexpr int kC4MergeTiles = 16;  // tiles of weights a block takes at once: 16 threads a tile, 4 keys each
// Tiles' worth of time that a row costs a block that adds weights (the same calls with
// weights: 29.9 | 132.8 us; with 12 30.3 | 134.3, with 48 30.2 | 134.0).
constexpr int kC4MergeRowCost = 24;

// The CTAs that hold a segment of a row whose units begin at `start` of the list.
struct C4Parts {
  int first, count;
};
__device__ __forceinline__ C4Parts c4_parts(int64_t start, int nt, int64_t share) {
  C4Parts r;
  r.first = static_cast<int>((start + kC4RowCost) / share);
  r.count = nt == 0 ? 0 : static_cast<int>((start + kC4RowCost + nt - 1) / share) - r.first + 1;
  return r;
}

// Statistics of a row's partials, by one warp: the maximum and the sum
// relative to it (log2 units).
__device__ __forceinline__ float2 c4_join_stats(const float2* ml, int count, int lane) {
  const float2 f0 = lane < count ? __ldg(&ml[static_cast<int64_t>(lane) * kC4Heads]) : make_float2(-INFINITY, 0.f);
  float top = f0.x;
  for (int i = lane + 32; i < count; i += 32) top = fmaxf(top, __ldg(&ml[static_cast<int64_t>(i) * kC4Heads].x));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  float ls = fmaf(top == -INFINITY ? 0.f : ex2_approx(f0.x - top), f0.y, 0.f);
  for (int i = lane + 32; i < count; i += 32) {
    const float2 f = __ldg(&ml[static_cast<int64_t>(i) * kC4Heads]);
    ls = fmaf(top == -INFINITY ? 0.f : ex2_approx(f.x - top), f.y, ls);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, off);
  return make_float2(top, ls);
}

// Joins the partials of every (sequence, query head) into O and LSE, and adds
// each entry's attention weight, summed over the heads of its group, where
// the scores were kept.  `m.warps` (1, 2, 4, 8) warps share a row's partials,
// four of them in flight each: with one warp, the 77 partials of a row of
// 131072 keys took 33 us, most of it waiting for memory.  The first four are
// fetched while the statistics are joined (that call: 1.2 us less), and four
// blocks an SM hold 64 registers a thread (64 sequences of up to 16000 with
// weights: 2.4 us less than with 75).
template <int D, int kType, bool kWeight>
__global__ void __launch_bounds__(kC4MergeThreads, 4) attn_cache4_merge_kernel(const DecMergeParams m) {
  constexpr int kWarps = kC4MergeThreads / 32;
  constexpr int kPer = D / 32;
  using Vec = typename std::conditional<kPer == 4, float4, float2>::type;
  const DecParams& p = m.d;
  __shared__ int64_t sums_s[kWarps];
  __shared__ int64_t before_s;
  __shared__ int b_s;
  __shared__ float lse_s[128];
  __shared__ __align__(16) float o_s[kWarps][D];
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  // The lengths are read before the wait, while the decode kernel finishes.  What
  // wrote them is complete: this kernel starts when every kernel before it in the
  // stream has started and let it, and the decode kernel of the same call is one of
  // them, whose blocks let it only after their own wait.  That holds with launches
  // of other threads in between, too; only a launch that writes these lengths may
  // not come there, as nothing may that writes the cache during the call.
  int64_t mine_before, mine;
  const int rows_per_b = p.c.H * p.HB;
  const int64_t count = c4_total(p, sums_s, &mine_before, &mine);
  // Weights: the tiles of every (sequence, key head) in equal contiguous
  // shares, one for each of the first blocks, walked row by row.  The share's
  // first row is found now, too (32 sequences of up to 4001: 0.6 us less).
  C4Walk w;
  w.x = w.end = 0;
  if (kWeight && blockIdx.x < m.weight_blocks) {
    const int64_t all = c4_units(count, kC4MergeRowCost) * p.c.H;
    const int64_t mine_w = (all + m.weight_blocks - 1) / m.weight_blocks;
    w.x = blockIdx.x * mine_w;
    w.end = w.x + mine_w < all ? w.x + mine_w : all;
    if (w.x < w.end) c4_find(p, w.x / p.c.H, kC4MergeRowCost, mine_before, mine, &b_s, &before_s);
  }
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t share = max(static_cast<int64_t>(1), (c4_units(count, kC4RowCost) * rows_per_b + m.dec_grid - 1) / m.dec_grid);

  // O and LSE: m.warps warps a row, the blocks' rows all of one sequence.
  const int hq = p.c.H * p.G, rows = kWarps / m.warps;
  const int per_b = (hq + rows - 1) / rows;
  const unsigned row_block = blockIdx.x - (kWeight ? m.weight_blocks : 0u), row_blocks = gridDim.x - (kWeight ? m.weight_blocks : 0u);
  for (int64_t u = row_block; u < static_cast<int64_t>(p.B) * per_b && (!kWeight || blockIdx.x >= m.weight_blocks); u += row_blocks) {
    const int b = static_cast<int>(u / per_b);
    const int head = static_cast<int>(u % per_b) * rows + warp / m.warps;
    const int stripe = (p.B + kC4MergeThreads - 1) / kC4MergeThreads;
    if (b / stripe == tid) {  // what lies before sequence b: its stripe's owner knows
      int64_t at = mine_before;
      for (int i = tid * stripe; i < b; ++i) at += c4_count(c4_tiles(p, i));
      before_s = at;
    }
    __syncthreads();
    const int64_t before = c4_units(before_s, kC4RowCost) * rows_per_b;
    float acc[kPer], inv = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
    const int64_t row = static_cast<int64_t>(b) * hq + head;
    if (head < hq) {
      const int h = head / p.G, g = head % p.G, hb = g / kC4Heads;
      const int in_b = h * p.HB + hb;
      const int nt = c4_tiles(p, b);
      const C4Parts cut = c4_parts(before + static_cast<int64_t>(in_b) * c4_row_units(nt, kC4RowCost), nt, share);
      const int64_t slot0 = cut.first + static_cast<int64_t>(b) * rows_per_b + in_b;
      const float2* ml = p.ml_part + slot0 * kC4Heads + g % kC4Heads;
      const float* op = p.o_part + (slot0 * kC4Heads + g % kC4Heads) * D + lane * kPer;
      const int step = m.warps;
      // the first partials come while the statistics are joined
      Vec v[4];
      float a[4];
      const auto load = [&](int i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t at = min(i + j * step, cut.count - 1);
          v[j] = __ldg(reinterpret_cast<const Vec*>(op + at * kC4Heads * D));
          a[j] = __ldg(&ml[at * kC4Heads].x);
        }
      };
      int i = warp % step;
      if (i < cut.count) load(i);
      const float2 tl = c4_join_stats(ml, cut.count, lane);
      inv = cut.count == 0 ? 0.f : 1.f / tl.y;
      while (i < cut.count) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (i + j * step >= cut.count) break;
          const float w = tl.x == -INFINITY ? 0.f : ex2_approx(a[j] - tl.x);
          const float* f = reinterpret_cast<const float*>(&v[j]);
#pragma unroll
          for (int e = 0; e < kPer; ++e) acc[e] = fmaf(w, f[e], acc[e]);
        }
        i += 4 * step;
        if (i < cut.count) load(i);
      }
      if (lane == 0 && warp % step == 0) p.lse[row] = cut.count == 0 ? -INFINITY : (tl.x + log2f(tl.y)) * kLn2;
    }
    if (m.warps > 1) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) o_s[warp][lane * kPer + e] = acc[e];
      __syncthreads();
      if (warp % m.warps == 0)
        for (int w = 1; w < m.warps; ++w)
#pragma unroll
          for (int e = 0; e < kPer; ++e) acc[e] += o_s[warp + w][lane * kPer + e];
    }
    if (head < hq && warp % m.warps == 0) {
      uint16_t* dst = p.o + row * D + lane * kPer;
      const uint32_t lo = pack_16x2<kType>(acc[0] * inv, acc[1] * inv);
      if constexpr (kPer == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(lo, pack_16x2<kType>(acc[2] * inv, acc[3] * inv));
      else
        *reinterpret_cast<uint32_t*>(dst) = lo;
    }
    __syncthreads();
  }

  if constexpr (kWeight) {
    if (w.x < w.end) {
      __syncthreads();
      w.b = b_s;
      w.before = before_s;
      while (w.next(p, p.c.H, kC4MergeRowCost)) {
        const int b = w.b, n = w.n, nt = w.nt, h = w.row;
        const int64_t before = c4_units(w.before, kC4RowCost) * rows_per_b;
        // log2 of the sum of every head of the group, a warp a head
        for (int g = warp; g < p.G; g += kWarps) {
          const int in_b = h * p.HB + g / kC4Heads;
          const C4Parts cut = c4_parts(before + static_cast<int64_t>(in_b) * c4_row_units(nt, kC4RowCost), nt, share);
          const int64_t slot0 = cut.first + static_cast<int64_t>(b) * rows_per_b + in_b;
          const float2 tl = c4_join_stats(p.ml_part + slot0 * kC4Heads + g % kC4Heads, cut.count, lane);
          if (lane == 0) lse_s[g] = tl.x + log2f(tl.y);
        }
        __syncthreads();
        c4_add_weights<false>(p, b, h, n, w.t0, w.t1, p.scores + ((w.before & kC4Tiles) * p.c.H + static_cast<int64_t>(h) * nt) * p.G * kC4TileKeys,
                              lse_s);
        __syncthreads();
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Eviction by accumulated attention weight
// ---------------------------------------------------------------------------
//
// Of the n entries of one (sequence, key head), `left` = min(n, budget) stay:
// first the protected ones (position > newest position - recent), then those
// of the highest weight, ties to the lower slot.  Kept entries at slots >=
// left move into the slots < left of the others, the i-th of the first to the
// i-th of the second.  So an entry moves at most once, every source lies at or
// behind `left` and every target before it, and nothing is read that the call
// writes.
//
// One thread-block cluster per (sequence, key head): each CTA holds a slice of
// the slots' rank keys in shared memory.  The left-th largest key is found by
// a radix select, 8 bits a round, most significant first, over histograms
// that the CTAs add up through distributed shared memory; counts of ties,
// holes and movers before each slice come the same way.  Every key is read
// from HBM once, whatever the budget.  A CTA of a long row (8192 entries to
// 2048) needs 23 us: 2 to read weights and positions, 1 for the protected ones,
// 3 for the radix rounds, 4 for ranks and lists, and 12 for its 1562 moves of 288
// bytes, which is what one SM can move; 24 sequences of 8 heads take 25 us.

// Threads of a CTA.  1024 hide more of the latency of long slices and many moves
// (24 sequences of up to 8192 entries cut to 2048: 26 us against 37 us with 512),
// but an SM's registers hold one such CTA: where the slices are short, two of
// 512 are faster (32 sequences of 2049 cut to 2048: 11 us against 20 us).
constexpr int kC4EvictFew = 512, kC4EvictMany = 1024;
constexpr int kC4EvictLong = 4096;  // a slice of more entries takes kC4EvictMany threads
constexpr int kC4EvictCluster = 8;             // CTAs of a cluster at most
constexpr int kC4EvictSmemKeys = 48 * 1024;    // keys a CTA can hold in shared memory: its slice at most

struct EvictParams {
  Cache4 c;
  const float* w_in;
  const int32_t* p_in;
  const int32_t* len;
  float* w_out;
  int32_t* p_out;
  int32_t* len_out;  // null: another launch writes the lengths
  int most;          // bound on the lengths
  int budget;
  int recent;
  int32_t* moves;    // [B*H][2][list]: holes, then movers
  int list;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// 32-bit load from the same shared-memory variable of another CTA of the cluster
__device__ __forceinline__ uint32_t ld_cluster_u32(const void* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Order of the weights as unsigned integers: NaN above +inf, -0 equal to +0;
// the protected entries above them all.
constexpr uint32_t kC4Protected = 0xffffffffu;
__device__ __forceinline__ uint32_t c4_rank_key(float w) {
  if (w != w) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sums over the block's table of `n` <= 2 * kThreads counts, in place;
// returns the total.  Two 16-bit counts share a word (sums below 2^16).
template <int kThreads>
__device__ __forceinline__ uint32_t block_scan(uint32_t* table, int n, uint32_t* warp_s) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const uint32_t v0 = 2 * tid < n ? table[2 * tid] : 0u, v1 = 2 * tid + 1 < n ? table[2 * tid + 1] : 0u;
  uint32_t incl = v0 + v1;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) warp_s[warp] = incl;
  __syncthreads();
  uint32_t ws = lane < kThreads / 32 ? warp_s[lane] : 0u;  // every warp sums the warps' totals
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, ws, off);
    if (lane >= off) ws += y;
  }
  const uint32_t total = __shfl_sync(0xffffffffu, ws, kThreads / 32 - 1);
  const uint32_t before = warp > 0 ? __shfl_sync(0xffffffffu, ws, warp - 1) : 0u;
  const uint32_t excl = before + incl - v0 - v1;
  if (2 * tid < n) table[2 * tid] = excl;
  if (2 * tid + 1 < n) table[2 * tid + 1] = excl + v0;
  __syncthreads();
  return total;
}

// kMulti: clusters of more than one CTA; without, the cluster barriers are the
// block's own.
template <int D, bool kMulti, int kThreads>
__global__ void __launch_bounds__(kThreads) attn_cache4_evict_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint32_t smem_keys[];
  __shared__ uint32_t hist[2][256];  // rounds alternate, so that one is cleared while the other is read
  __shared__ uint32_t sums[kMulti ? 256 : 1];
  __shared__ uint32_t share[4];      // what the other CTAs read: newest, ties, holes, movers
  __shared__ uint32_t found[3];      // digit, entries still to take, entries with it
  __shared__ uint32_t warp_s[kThreads / 32];
  // of each warp's 32 slots in each round over the slice: ties, or holes and movers
  constexpr int kWarps = kThreads / 32;
  __shared__ uint32_t table[kThreads == kC4EvictMany ? 2 * kThreads : (kC4EvictLong / kThreads + 1) * kWarps];
  static_assert(kThreads != kC4EvictMany || kC4EvictSmemKeys / 32 <= 2 * kThreads, "the table holds a slice in shared memory");
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  const uint32_t rank = kMulti ? cluster_rank() : 0u, R = kMulti ? cluster_size() : 1u;
  const auto sync_all = [] {
    if constexpr (kMulti)
      cluster_sync_all();
    else
      __syncthreads();
  };
  const auto peer = [](const uint32_t* v, uint32_t q) { return kMulti ? ld_cluster_u32(v, q) : *static_cast<const volatile uint32_t*>(v); };
  const int64_t bh = blockIdx.x / R;
  const int b = static_cast<int>(bh / p.c.H);
  if (tid < 256) hist[0][tid] = hist[1][tid] = 0u;
  grid_dependency_wait();
  const int n = c4_len(p.len, b, p.most);
  const int left = min(n, p.budget);
  const int64_t base = bh * p.c.cap;
  if (p.len_out != nullptr && bh % p.c.H == 0 && rank == 0 && tid == 0) p.len_out[b] = left;
  const int slice = (n + static_cast<int>(R) - 1) / static_cast<int>(R);
  const int i0 = min(n, static_cast<int>(rank) * slice), i1 = min(n, i0 + slice), mine = i1 - i0;
  const float* const w_in = p.w_in + base + i0;
  const int32_t* const p_in = p.p_in + base + i0;
  const bool copy_w = p.w_out != p.w_in, copy_p = p.p_out != p.p_in;
  if (n <= p.budget) {  // every entry stays where it is (the same for the whole cluster)
    for (int i = tid; i < mine; i += kThreads) {
      if (copy_w) p.w_out[base + i0 + i] = w_in[i];
      if (copy_p) p.p_out[base + i0 + i] = p_in[i];
    }
    grid_launch_dependents();
    return;
  }
  uint32_t* const key = smem_keys;

  // Rank keys of the slice, and the newest position; four entries in flight a
  // thread.
  constexpr int kU = 4;
  int newest = INT_MIN;
  for (int i = tid; i < mine; i += kU * kThreads) {
    float w[kU];
    int at[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int j = min(i + u * kThreads, mine - 1);
      w[u] = w_in[j];
      at[u] = p_in[j];
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      newest = max(newest, at[u]);
      if (i + u * kThreads < mine) key[i + u * kThreads] = c4_rank_key(w[u]);
    }
  }
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) warp_s[tid >> 5] = static_cast<uint32_t>(newest);
  __syncthreads();
  if (tid < 32) {
    newest = tid < kThreads / 32 ? static_cast<int>(warp_s[tid]) : INT_MIN;
    newest = __reduce_max_sync(0xffffffffu, newest);
    if (tid == 0) share[0] = static_cast<uint32_t>(newest);
  }
  sync_all();
  if (p.recent > 0) {
    newest = INT_MIN;
    for (uint32_t q = 0; q < R; ++q) newest = max(newest, static_cast<int>(peer(&share[0], q)));
    const int64_t old = static_cast<int64_t>(newest) - p.recent;
    for (int i = tid; i < mine; i += kU * kThreads) {
      int at[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) at[u] = p_in[min(i + u * kThreads, mine - 1)];
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (i + u * kThreads < mine && at[u] > old) key[i + u * kThreads] = kC4Protected;
    }
  }

  // The left-th largest key, digit by digit: `take` of the keys that agree with
  // `prefix` in the digits seen are kept, and all above.  It ends early where
  // all of them are (for weights that differ, mostly a digit early).
  uint32_t prefix = 0u, take = static_cast<uint32_t>(left), seen = 0u;
  bool ties = true;
  for (int round = 0; round < 4 && ties; ++round) {
    const int shift = 24 - 8 * round;
    uint32_t* const h = hist[round & 1];
    for (int i = tid; i < mine; i += kThreads) {
      const uint32_t k = key[i];
      if ((k & seen) == prefix) atomicAdd(&h[(k >> shift) & 255u], 1u);
    }
    sync_all();
    // the other histogram was read in the round before, by every CTA before the
    // barrier above
    if (tid >= kThreads - 256) hist[(round & 1) ^ 1][tid - (kThreads - 256)] = 0u;
    const uint32_t* bins = h;
    if constexpr (kMulti) {  // a thread a bin: each waits for R remote loads, not for 8 R
      if (tid < 256) {
        uint32_t sum = 0u;
        for (uint32_t q = 0; q < R; ++q) sum += peer(&h[tid], q);
        sums[tid] = sum;
      }
      __syncthreads();
      bins = sums;
    }
    if (tid < 32) {  // digits from the top: lane j has 255 - 8j .. 248 - 8j
      uint32_t cnt[8], sum = 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        cnt[e] = bins[255 - 8 * lane - e];
        sum += cnt[e];
      }
      uint32_t incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
      }
      uint32_t before = incl - sum;
      if (before < take && take <= incl) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (before < take && take <= before + cnt[e]) {
            found[0] = static_cast<uint32_t>(255 - 8 * lane - e);
            found[1] = take - before;
            found[2] = cnt[e];
          }
          before += cnt[e];
        }
      }
    }
    __syncthreads();
    prefix |= found[0] << shift;
    seen |= 255u << shift;
    take = found[1];
    ties = found[2] != take;
    __syncthreads();  // found may be written again
  }

  // Kept: keys above `prefix` in the digits seen, and the first `take` equal to
  // it, in slot order.  Ranks come from the warps' votes, a table of their
  // counts and its sums: three coalesced passes over the keys.
  const int warp = tid >> 5;
  const uint32_t below = (1u << lane) - 1u;
  const int rounds = (mine + kThreads - 1) / kThreads;
  uint32_t eq_before = 0u;  // ties in the slices before this one
  if (ties) {
    for (int j = 0; j < rounds; ++j) {
      const int i = j * kThreads + tid;
      const uint32_t eq = __ballot_sync(0xffffffffu, i < mine && (key[i] & seen) == prefix);
      if (lane == 0) table[j * kWarps + warp] = __popc(eq);
    }
    __syncthreads();
    const uint32_t all = block_scan<kThreads>(table, rounds * kWarps, warp_s);
    if (kMulti) {
      if (tid == 0) share[1] = all;
      sync_all();
      for (uint32_t q = 0; q < rank; ++q) eq_before += peer(&share[1], q);
    }
  }
  for (int j = 0; j < rounds; ++j) {
    const int i = j * kThreads + tid;
    bool keep = false;
    if (ties) {
      const bool eq = i < mine && (key[i] & seen) == prefix;
      const uint32_t votes = __ballot_sync(0xffffffffu, eq);
      if (eq) keep = eq_before + table[j * kWarps + warp] + __popc(votes & below) < take;
      __syncwarp();  // the table entry is read: it is written below
    } else if (i < mine) {
      keep = (key[i] & seen) == prefix;
    }
    if (i < mine) {
      keep = keep || (key[i] & seen) > prefix;
      key[i] = keep;
    }
    const uint32_t hole = __ballot_sync(0xffffffffu, i < mine && !keep && i0 + i < left);
    const uint32_t mover = __ballot_sync(0xffffffffu, i < mine && keep && i0 + i >= left);
    if (lane == 0) table[j * kWarps + warp] = __popc(hole) | __popc(mover) << 16;
  }
  __syncthreads();
  const uint32_t all = block_scan<kThreads>(table, rounds * kWarps, warp_s);
  uint32_t hole0 = 0u, mover0 = 0u, n_moves = all & 0xffffu;
  if (kMulti) {
    if (tid == 0) {
      share[2] = all & 0xffffu;
      share[3] = all >> 16;
    }
    sync_all();
    n_moves = 0u;
    for (uint32_t q = 0; q < R; ++q) {
      const uint32_t x = peer(&share[2], q);
      if (q < rank) {
        hole0 += x;
        mover0 += peer(&share[3], q);
      }
      n_moves += x;
    }
  }
  int32_t* const holes = p.moves + bh * 2 * p.list;
  int32_t* const movers = holes + p.list;
  for (int j = 0; j < rounds; ++j) {
    const int i = j * kThreads + tid;
    const bool keep = i < mine && key[i] != 0u;
    const bool is_hole = i < mine && !keep && i0 + i < left, is_mover = keep && i0 + i >= left;
    const uint32_t hole = __ballot_sync(0xffffffffu, is_hole), mover = __ballot_sync(0xffffffffu, is_mover);
    const uint32_t at = table[j * kWarps + warp];
    if (is_hole) holes[hole0 + (at & 0xffffu) + __popc(hole & below)] = i0 + i;
    if (is_mover) movers[mover0 + (at >> 16) + __popc(mover & below)] = i0 + i;
  }
  sync_all();  // the lists are written; no CTA reads another's shared memory any more
  grid_launch_dependents();
  if (copy_w || copy_p) {
    for (int i = tid; i < min(mine, left - i0); i += kThreads) {
      if (key[i] == 0u) continue;
      if (copy_w) p.w_out[base + i0 + i] = w_in[i];
      if (copy_p) p.p_out[base + i0 + i] = p_in[i];
    }
  }

  // The moves, 16 bytes a lane: half of a move's lanes take K, half V; four
  // moves in flight each.
  constexpr int kLanes = D / 16;
  constexpr int kWords = D / 32;  // 16-byte words of a row
  constexpr int kMeta = D / kC4Group;
  const int part = tid % kLanes, word = part % kWords;
  const bool is_v = part >= kWords;
  uint8_t* const codes = is_v ? p.c.v : p.c.k;
  using Meta = typename std::conditional<kMeta == 2, uint2, uint32_t>::type;  // a row's (s, m)
  Meta* const meta = reinterpret_cast<Meta*>(is_v ? p.c.vm : p.c.km);
  const uint32_t* const in = is_v ? reinterpret_cast<const uint32_t*>(p.p_in) : reinterpret_cast<const uint32_t*>(p.w_in);
  uint32_t* const out = is_v ? reinterpret_cast<uint32_t*>(p.p_out) : reinterpret_cast<uint32_t*>(p.w_out);
  const uint32_t step = R * (kThreads / kLanes);
  for (uint32_t m = rank * (kThreads / kLanes) + tid / kLanes; m < n_moves; m += kU * step) {
    int64_t to[kU], from[kU];
    uint4 x[kU];
    Meta sm[kU];
    uint32_t extra[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t j = min(m + u * step, n_moves - 1);
      to[u] = base + __ldcg(holes + j);
      from[u] = base + __ldcg(movers + j);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      x[u] = *(reinterpret_cast<const uint4*>(codes + from[u] * (D / 2)) + word);
      if (word == 0) {
        sm[u] = meta[from[u]];
        extra[u] = in[from[u]];
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (m + u * step >= n_moves) break;
      *(reinterpret_cast<uint4*>(codes + to[u] * (D / 2)) + word) = x[u];
      if (word == 0) {
        meta[to[u]] = sm[u];
        out[to[u]] = extra[u];
      }
    }
  }
}

// Lengths after an eviction, where they take the place of the old ones: a
// launch behind the one whose blocks read those.
__global__ void attn_cache4_cut_kernel(int32_t* len, int B, int most, int budget) {
  grid_dependency_wait();
  grid_launch_dependents();
  for (int64_t b = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; b < B;
       b += static_cast<int64_t>(gridDim.x) * blockDim.x)
    len[b] = min(min(max(len[b], 0), most), budget);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

using EvictKernel = void (*)(EvictParams);
// by D = 128, a cluster of several CTAs, long slices
constexpr EvictKernel kEvictKernels[8] = {
    attn_cache4_evict_kernel<64, false, kC4EvictFew>,  attn_cache4_evict_kernel<64, false, kC4EvictMany>,
    attn_cache4_evict_kernel<64, true, kC4EvictFew>,   attn_cache4_evict_kernel<64, true, kC4EvictMany>,
    attn_cache4_evict_kernel<128, false, kC4EvictFew>, attn_cache4_evict_kernel<128, false, kC4EvictMany>,
    attn_cache4_evict_kernel<128, true, kC4EvictFew>,  attn_cache4_evict_kernel<128, true, kC4EvictMany>};
std::atomic<int> g_cache4_state[kMaxDevices];  // 1: shared-memory limits set

attn_status_t prepare_cache4(int* dev, int* sms) {
  if (cudaGetDevice(dev) != cudaSuccess) return ATTN_ERR_DEVICE;
  const attn_status_t ps = prepare_device(*dev);
  if (ps != ATTN_OK) return ps;
  if (g_cache4_state[*dev].load(std::memory_order_acquire) == 0) {
    for (const EvictKernel k : kEvictKernels)
      if (cudaFuncSetAttribute(reinterpret_cast<const void*>(k), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kC4EvictSmemKeys * 4) != cudaSuccess)
        return ATTN_ERR_DEVICE;
    g_cache4_state[*dev].store(1, std::memory_order_release);
  }
  *sms = g_dev_sms[*dev].load(std::memory_order_relaxed);
  return ATTN_OK;
}

// The cache's own arguments (nothing is launched).
attn_status_t check_cache4(const attn_cache4_t* c) {
  if (c == nullptr || c->B < 1 || c->H_kv < 1 || c->capacity < 1) return ATTN_ERR_INVALID_ARG;
  if (c->k_codes == nullptr || c->k_meta == nullptr || c->v_codes == nullptr || c->v_meta == nullptr ||
      c->length == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return ATTN_ERR_UNSUPPORTED;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_meta, 8) || !aligned(c->v_meta, 8) ||
      !aligned(c->length, 4) || !aligned(c->weight, 4) || !aligned(c->pos, 4))
    return ATTN_ERR_ALIGNMENT;
  if (static_cast<int64_t>(c->B) * c->H_kv > INT_MAX / 64) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

Cache4 cache4_of(const attn_cache4_t* c) {
  Cache4 r;
  r.k = static_cast<uint8_t*>(c->k_codes);
  r.v = static_cast<uint8_t*>(c->v_codes);
  r.km = static_cast<uint32_t*>(c->k_meta);
  r.vm = static_cast<uint32_t*>(c->v_meta);
  r.H = c->H_kv;
  r.cap = c->capacity;
  return r;
}

// Packed rows of K and V: sizes, strides, alignment to 8 elements.
attn_status_t check_rows(const attn_cache4_t* c, const void* k, const void* v, int64_t rows, int64_t k_stride,
                         int64_t v_stride, const int32_t* seq_start, int elem_bytes) {
  if (rows < 0) return ATTN_ERR_INVALID_ARG;
  if (seq_start == nullptr && rows != c->B) return ATTN_ERR_INVALID_ARG;
  if (rows > 0 && (k == nullptr || v == nullptr)) return ATTN_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(c->H_kv) * c->D;
  if (k_stride < row || v_stride < row) return ATTN_ERR_INVALID_ARG;
  const int64_t unit = 16 / elem_bytes;
  if (!aligned(k, 16) || !aligned(v, 16) || k_stride % unit != 0 || v_stride % unit != 0 || !aligned(seq_start, 4))
    return ATTN_ERR_ALIGNMENT;
  if (rows > INT_MAX) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// Key heads a block walks, so that there are four blocks an SM or a block for
// every key head, and the grid: runs of key heads x chunks of rows.
struct RowsGrid {
  int heads;
  dim3 grid;
};
RowsGrid rows_grid(int64_t rows, int D, int H, int sms) {
  const int64_t block_rows = D == 64 ? kC4BlockRows<64> : kC4BlockRows<128>;
  const int64_t chunks = std::max<int64_t>(1, std::min<int64_t>((rows + block_rows - 1) / block_rows, 65535));
  const int64_t runs = std::min<int64_t>(H, std::max<int64_t>(1, (4 * sms + chunks - 1) / chunks));
  RowsGrid r;
  r.heads = static_cast<int>((H + runs - 1) / runs);
  r.grid = dim3(static_cast<unsigned>((H + r.heads - 1) / r.heads), static_cast<unsigned>(chunks));
  return r;
}

// One CTA a row; the workspace then holds the scores of a call with weights.
bool decode_direct(int max_len, int HB, bool weight) {
  return max_len <= kC4DirectLen && (HB == 1 || !weight);
}

// Workspace of a decode call: partial O, partial (m, l), and with weights the
// scores of every tile.
struct DecLayout {
  int64_t slots, o_bytes, ml_bytes, score_bytes;
  int grid;
};
DecLayout decode_layout(int B, int H_q, int H_kv, int D, int max_len, bool weight, int sms) {
  const int64_t G = H_q / H_kv, HB = (G + kC4Heads - 1) / kC4Heads;
  const int64_t rows = static_cast<int64_t>(B) * H_kv * HB;
  const int64_t tiles = (static_cast<int64_t>(max_len) + kC4TileKeys - 1) / kC4TileKeys;
  DecLayout l;
  l.grid = static_cast<int>(std::min<int64_t>(rows * (tiles + kC4RowCost), static_cast<int64_t>(sms) * kC4DecCtasPerSm));
  l.slots = l.grid + rows;
  l.o_bytes = l.slots * kC4Heads * D * 4;
  l.ml_bytes = l.slots * kC4Heads * 8;
  l.score_bytes = weight ? static_cast<int64_t>(B) * H_kv * tiles * G * kC4TileKeys * 4 : 0;
  return l;
}

template <int D, int kType>
attn_status_t launch_decode(DecMergeParams m, int sms, cudaStream_t stream) {
  const bool weight = m.d.w_out != nullptr;
  if (decode_direct(m.d.most, m.d.HB, weight)) {
    const dim3 rows(static_cast<unsigned>(m.d.B * m.d.c.H * m.d.HB));
    const cudaError_t e =
        weight ? launch_pdl(attn_cache4_decode_kernel<D, kType, true, true>, rows, dim3(kC4DecThreads), 0, stream, m.d)
               : launch_pdl(attn_cache4_decode_kernel<D, kType, false, true>, rows, dim3(kC4DecThreads), 0, stream, m.d);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
  }
  const dim3 grid(static_cast<unsigned>(m.dec_grid));
  cudaError_t e = weight ? launch_pdl(attn_cache4_decode_kernel<D, kType, true, false>, grid, dim3(kC4DecThreads), 0, stream, m.d)
                         : launch_pdl(attn_cache4_decode_kernel<D, kType, false, false>, grid, dim3(kC4DecThreads), 0, stream, m.d);
  if (e != cudaSuccess) return ATTN_ERR_LAUNCH;
  const int64_t rows = kC4MergeThreads / 32 / m.warps;
  const int64_t tiles = (static_cast<int64_t>(m.d.most) + kC4TileKeys - 1) / kC4TileKeys * m.d.B * m.d.c.H;
  // Three blocks an SM for the weights, of the four that fit: a block's set-up is
  // some 700 instructions a warp, ten times a tile's.  (32 sequences of up to 4001
  // and 64 of up to 16000: with four 0.4 and 0.5 us more, with eight behind the
  // rows' blocks 3.0 and 3.6.)
  const int64_t row_blocks = std::min<int64_t>(m.d.B * ((static_cast<int64_t>(m.d.c.H) * m.d.G + rows - 1) / rows),
                                               static_cast<int64_t>(sms) * 4);
  m.weight_blocks =
      weight ? static_cast<unsigned>(std::min<int64_t>((tiles + kC4MergeTiles - 1) / kC4MergeTiles, static_cast<int64_t>(sms) * 3)) : 0u;
  const dim3 mg(static_cast<unsigned>(row_blocks) + m.weight_blocks);
  e = weight ? launch_pdl(attn_cache4_merge_kernel<D, kType, true>, mg, dim3(kC4MergeThreads), 0, stream, m)
             : launch_pdl(attn_cache4_merge_kernel<D, kType, false>, mg, dim3(kC4MergeThreads), 0, stream, m);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

// CTAs of an eviction's clusters: enough to give every SM one, with slices of
// at least 1024 entries; or as many as hold the keys in shared memory.  More
// clusters than that lose: with pairs for 256 rows of 2049 entries a call took
// 27 us instead of 11, for 192 rows of up to 8192 28 instead of 25 (fours: 39).
int evict_cluster(int64_t BH, int max_len) {
  int R = 1;
  while (R < kC4EvictCluster && ((BH * R < kC4WorkspaceSms && max_len / (2 * R) >= 1024) || max_len > R * kC4EvictSmemKeys)) R *= 2;
  return R;
}
int64_t evict_list(int max_len, int budget) {
  return std::max<int64_t>(1, std::min<int64_t>(budget, static_cast<int64_t>(max_len) - budget));
}
// Longest sequences whose keys a cluster holds.
constexpr int kC4EvictMostLen = kC4EvictCluster * kC4EvictSmemKeys;
static_assert(kC4EvictMostLen == ATTN_CACHE4_EVICT_MAX_LEN, "the header's limit");

}  // namespace

extern "C" {

attn_status_t attn_cache4_append(const attn_cache4_t* cache, const void* k, const void* v, int64_t rows,
                                 int64_t k_stride, int64_t v_stride, int dtype, const int32_t* seq_start,
                                 const int32_t* first_pos, int32_t* length_out, void* stream) {
  attn_status_t st = check_cache4(cache);
  if (st != ATTN_OK) return st;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16) return ATTN_ERR_UNSUPPORTED;
  st = check_rows(cache, k, v, rows, k_stride, v_stride, seq_start, 2);
  if (st != ATTN_OK) return st;
  if (length_out == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!aligned(first_pos, 4) || !aligned(length_out, 4)) return ATTN_ERR_ALIGNMENT;
  int dev = 0, sms = 0;
  st = prepare_cache4(&dev, &sms);
  if (st != ATTN_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Cache4 c = cache4_of(cache);
  const Cache4Rows g{seq_start, cache->length, cache->B, rows, k_stride, v_stride};
  const bool in_place = length_out == cache->length;
  int32_t* const len_out = in_place ? nullptr : length_out;
  const uint16_t* k16 = static_cast<const uint16_t*>(k);
  const uint16_t* v16 = static_cast<const uint16_t*>(v);
  const RowsGrid rg = rows_grid(rows, cache->D, c.H, sms);
  const auto run = [&](auto kernel) {
    return launch_pdl(kernel, rg.grid, dim3(kC4RowsThreads), 0, s, k16, v16, g, c, rg.heads, cache->weight, cache->pos,
                      first_pos, len_out);
  };
  cudaError_t e;
  if (cache->D == 64)
    e = dtype == ATTN_BF16 ? run(attn_cache4_append_kernel<64, kBF16>) : run(attn_cache4_append_kernel<64, kFP16>);
  else
    e = dtype == ATTN_BF16 ? run(attn_cache4_append_kernel<128, kBF16>) : run(attn_cache4_append_kernel<128, kFP16>);
  if (e == cudaSuccess && in_place)
    e = launch_pdl(attn_cache4_grow_kernel, dim3(static_cast<unsigned>(std::min((cache->B + 255) / 256, 64))), dim3(256), 0, s, g,
                   length_out, cache->capacity);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

attn_status_t attn_cache4_read(const attn_cache4_t* cache, void* k, void* v, int64_t rows, int64_t k_stride,
                               int64_t v_stride, int dtype, const int32_t* seq_start, const int32_t* first_slot,
                               void* stream) {
  attn_status_t st = check_cache4(cache);
  if (st != ATTN_OK) return st;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16 && dtype != ATTN_FP32) return ATTN_ERR_UNSUPPORTED;
  st = check_rows(cache, k, v, rows, k_stride, v_stride, seq_start, dtype == ATTN_FP32 ? 4 : 2);
  if (st != ATTN_OK) return st;
  if (!aligned(first_slot, 4)) return ATTN_ERR_ALIGNMENT;
  if (rows == 0) return ATTN_OK;
  int dev = 0, sms = 0;
  st = prepare_cache4(&dev, &sms);
  if (st != ATTN_OK) return st;
  const Cache4 c = cache4_of(cache);
  const Cache4Rows g{seq_start, first_slot, cache->B, rows, k_stride, v_stride};
  const RowsGrid rg = rows_grid(rows, cache->D, c.H, sms);
  const auto run = [&](auto kernel) {
    return launch_pdl(kernel, rg.grid, dim3(kC4RowsThreads), 0, static_cast<cudaStream_t>(stream), k, v, g, c, rg.heads);
  };
  cudaError_t e;
  if (cache->D == 64)
    e = dtype == ATTN_BF16   ? run(attn_cache4_read_kernel<64, kBF16>)
        : dtype == ATTN_FP16 ? run(attn_cache4_read_kernel<64, kFP16>)
                             : run(attn_cache4_read_kernel<64, kFP32>);
  else
    e = dtype == ATTN_BF16   ? run(attn_cache4_read_kernel<128, kBF16>)
        : dtype == ATTN_FP16 ? run(attn_cache4_read_kernel<128, kFP16>)
                             : run(attn_cache4_read_kernel<128, kFP32>);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

uint64_t attn_cache4_decode_workspace_bytes(int B, int H_q, int H_kv, int D, int max_len, int with_weight) {
  if (B < 1 || H_kv < 1 || H_q < H_kv || H_q % H_kv != 0 || H_q / H_kv > 128 || (D != 64 && D != 128) || max_len < 1)
    return 0;
  if (with_weight == 0 && decode_direct(max_len, 1, false)) return 16;
  const DecLayout l = decode_layout(B, H_q, H_kv, D, max_len, with_weight != 0, kC4WorkspaceSms);
  return static_cast<uint64_t>(l.o_bytes + l.ml_bytes + l.score_bytes);
}

attn_status_t attn_cache4_decode(const attn_cache4_t* cache, const void* q, int64_t q_stride, void* o, float* lse, int H_q,
                                 int dtype, float scale, int max_len, const float* weight_in, float* weight_out,
                                 void* workspace, uint64_t workspace_bytes, void* stream) {
  attn_status_t st = check_cache4(cache);
  if (st != ATTN_OK) return st;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16) return ATTN_ERR_UNSUPPORTED;
  if (q == nullptr || o == nullptr || lse == nullptr) return ATTN_ERR_INVALID_ARG;
  if (H_q < cache->H_kv || H_q % cache->H_kv != 0) return ATTN_ERR_INVALID_ARG;
  if (H_q / cache->H_kv > 128) return ATTN_ERR_UNSUPPORTED;
  if (q_stride < static_cast<int64_t>(H_q) * cache->D) return ATTN_ERR_INVALID_ARG;
  if (max_len < 1 || max_len > cache->capacity) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if ((weight_in == nullptr) != (weight_out == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || q_stride % 8 != 0 || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 16) ||
      !aligned(weight_in, 4) || !aligned(weight_out, 4))
    return ATTN_ERR_ALIGNMENT;
  if ((weight_out != nullptr || !decode_direct(max_len, 1, false)) &&
      (workspace == nullptr ||
       workspace_bytes < attn_cache4_decode_workspace_bytes(cache->B, H_q, cache->H_kv, cache->D, max_len, weight_out != nullptr)))
    return ATTN_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  st = prepare_cache4(&dev, &sms);
  if (st != ATTN_OK) return st;
  sms = std::min(sms, kC4WorkspaceSms);
  const DecLayout l = decode_layout(cache->B, H_q, cache->H_kv, cache->D, max_len, weight_out != nullptr, sms);
  DecMergeParams m;
  m.d.c = cache4_of(cache);
  m.d.q = static_cast<const uint16_t*>(q);
  m.d.q_stride = q_stride;
  m.d.len = cache->length;
  m.d.B = cache->B;
  m.d.G = H_q / cache->H_kv;
  m.d.HB = (m.d.G + kC4Heads - 1) / kC4Heads;
  m.d.most = max_len;
  m.d.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  char* ws = static_cast<char*>(workspace);
  m.d.o_part = reinterpret_cast<float*>(ws);
  m.d.ml_part = reinterpret_cast<float2*>(ws + l.o_bytes);
  m.d.scores = weight_out != nullptr ? reinterpret_cast<float*>(ws + l.o_bytes + l.ml_bytes) : nullptr;
  m.dec_grid = l.grid;
  m.d.o = static_cast<uint16_t*>(o);
  m.d.lse = lse;
  m.d.w_in = weight_in;
  m.d.w_out = weight_out;
  // a warp for every four partials that a row has on average
  const int64_t parts = l.grid / (static_cast<int64_t>(m.d.B) * m.d.c.H * m.d.HB) + 1;
  m.warps = parts > 16 ? 8 : parts > 8 ? 4 : parts > 4 ? 2 : 1;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cache->D == 64)
    return dtype == ATTN_BF16 ? launch_decode<64, kBF16>(m, sms, s) : launch_decode<64, kFP16>(m, sms, s);
  return dtype == ATTN_BF16 ? launch_decode<128, kBF16>(m, sms, s) : launch_decode<128, kFP16>(m, sms, s);
}

uint64_t attn_cache4_evict_workspace_bytes(int B, int H_kv, int max_len, int budget) {
  if (B < 1 || H_kv < 1 || max_len < 1 || budget < 1) return 0;
  if (budget >= max_len) return 16;
  if (max_len > kC4EvictMostLen) return 0;
  const int64_t BH = static_cast<int64_t>(B) * H_kv;
  return static_cast<uint64_t>(BH * 2 * evict_list(max_len, budget) * 4);
}

attn_status_t attn_cache4_evict(const attn_cache4_t* cache, int budget, int recent, int max_len, float* weight_out,
                                int32_t* pos_out, int32_t* length_out, void* workspace, uint64_t workspace_bytes,
                                void* stream) {
  attn_status_t st = check_cache4(cache);
  if (st != ATTN_OK) return st;
  if (cache->weight == nullptr || cache->pos == nullptr || weight_out == nullptr || pos_out == nullptr ||
      length_out == nullptr || workspace == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (budget < 1 || recent < 0 || recent > budget || max_len < 1 || max_len > cache->capacity) return ATTN_ERR_INVALID_ARG;
  if (max_len > kC4EvictMostLen && budget < max_len) return ATTN_ERR_UNSUPPORTED;
  if (!aligned(weight_out, 4) || !aligned(pos_out, 4) || !aligned(length_out, 4) || !aligned(workspace, 16))
    return ATTN_ERR_ALIGNMENT;
  if (workspace_bytes < attn_cache4_evict_workspace_bytes(cache->B, cache->H_kv, max_len, budget)) return ATTN_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  st = prepare_cache4(&dev, &sms);
  if (st != ATTN_OK) return st;
  const int64_t BH = static_cast<int64_t>(cache->B) * cache->H_kv;
  const int R = evict_cluster(BH, max_len);
  const bool in_place = length_out == cache->length;
  EvictParams p;
  p.c = cache4_of(cache);
  p.w_in = cache->weight;
  p.p_in = cache->pos;
  p.len = cache->length;
  p.w_out = weight_out;
  p.p_out = pos_out;
  p.len_out = in_place ? nullptr : length_out;
  p.most = max_len;
  p.budget = budget;
  p.recent = recent;
  p.list = budget < max_len ? static_cast<int>(evict_list(max_len, budget)) : 1;
  p.moves = static_cast<int32_t*>(workspace);
  const int slice = (max_len + R - 1) / R;
  const size_t smem = budget < max_len ? static_cast<size_t>(slice) * 4 : 16;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(R);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(BH * R));
  const bool many = slice > kC4EvictLong;
  cfg.blockDim = dim3(many ? kC4EvictMany : kC4EvictFew);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = R > 1 ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kEvictKernels[(cache->D == 128 ? 4 : 0) + (R > 1 ? 2 : 0) + (many ? 1 : 0)], p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess && in_place)
    e = launch_pdl(attn_cache4_cut_kernel, dim3(static_cast<unsigned>(std::min((cache->B + 255) / 256, 64))), dim3(256), 0, s,
                   length_out, cache->B, max_len, budget);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

}  // extern "C"
