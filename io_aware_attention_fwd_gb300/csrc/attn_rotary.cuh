// The norm of every query and key head and the rotation by its token's
// position, in one pass, with its gradient.  Part of attn_fwd.cu.
//
// For a head's row x of D channels, with weight w and position p:
//     r = 1 / sqrt(mean(x^2) + eps),  y = r w x,
//     (a, b) of pair i  ->  amplitude * (a cos t - b sin t, a sin t + b cos t),  t = p f_i,
// where pair i of the first `rot` channels is (i, i + rot/2), or (2i, 2i + 1)
// interleaved.  The gradient, from dy of the result: g = dy turned by -t,
//     dw = sum over tokens and heads of g r x,  dx = r (g w - r x mean(g w r x)).
//
// Angles.  A position times a frequency has to be known modulo one turn.  In
// fp32 a product of 10^5 radians is off by 2^-8; so frequencies are held as 64-bit
// fractions of a turn a position, f / (2 pi) * 2^64, and the product with an int
// modulo 2^64 is the angle to 2^-64 p of a turn: one integer multiplication.  Its
// upper 32 bits, as a signed number of half turns, go through sincospif.
//
// Both passes are bound by HBM: 4 (forward) or 6 (gradient) bytes a channel.
// A row of 256 (128) bytes is 16 (8) lanes of 8 channels, so a warp takes 2 (4) heads
// of a token at once; what pairs with a lane's channels is one shuffle of the 16-bit
// words away.  All groups of heads of all tokens form one list, cut into equal
// shares, one a warp, which has a few groups on their way, copied asynchronously into a
// ring of its own in shared memory (each lane its own 16 bytes).  The sine and cosine of a
// token are worked out by the warp that comes to it, while its first groups travel;
// what they and the weights make of a lane's channels,
//     y = r (x A + x' B)   (x' the paired channels),
// stays in registers for all heads of the token.
// 16384 tokens of 64 heads, D = 128 (537 MB): 87 us, 6.2 TB/s, against 86 us for a copy
// of the same tensors.  With a block's tokens' tables in shared memory, read for each
// head, it took 186 us; walking group by group with the addresses worked out anew, 159
// (226 instructions a group); four groups at once in registers, 96.  The gradient of as
// many tokens of 40 heads (503 MB): 104 us, 4.8 TB/s; it is held up by its 128 registers
// a thread (two blocks an SM), but three blocks spill and take 128 to 138.

namespace {

constexpr int kRotThreads = 256;
constexpr int kRotWarps = kRotThreads / 32;
constexpr int kRotFwdBlocks = 3;  // blocks an SM

struct RotRows {  // rows [B][S][H][D], strides in elements
  uint16_t* p;
  int64_t b, row, head;
};

struct RotTurn {
  const int64_t* turns;  // [rot / 2]
  int rot, inter;
  float amp;
};

struct RotParams {
  RotRows in[3];   // q, k; append: v too
  RotRows out[3];  // append: q alone, the others go to the pages
  RotRows dy[2];   // gradient
  int heads[3];
  int first[4];    // first group of q, k, v in a token's list, and their number
  const void* w[2];  // weights, or null: no norm
  int w_fp32;
  float eps;
  RotTurn turn;
  const int32_t* pos;  // [B][S]
  int S;
  int64_t total, share;  // groups of all tokens; of a warp
  float* dw;       // gradient: [blocks][2][D]
};

// What a lane holds of a row.
template <int D>
struct RotLane {
  static constexpr int kLanes = D / 8;       // lanes a row
  static constexpr int kRows = 32 / kLanes;  // rows a warp
  int sub, c0;                               // this lane's row of the warp's, and first channel
  int pair;                                  // where the paired channels are: a lane (half layout), or bytes of the same word
  bool turned, low;
  int at;                                    // of its first cosine
  __device__ RotLane(int lane, const RotTurn& t) {
    sub = lane / kLanes;
    c0 = (lane % kLanes) * 8;
    const int half = t.rot / 2;
    turned = c0 < t.rot;
    low = c0 < half;
    pair = t.inter ? (turned ? 0x1032 : 0x3210) : !turned ? lane : lane + (low ? half : -half) / 8;
    at = t.inter ? c0 / 2 : low ? c0 : c0 - half;
  }
};

// This lane's share of a token's cosines and sines, cs[0 .. rot/2 - 1] and behind them.
struct RotTable {
  int64_t turn[2];  // of pairs lane and lane + 32
  __device__ RotTable(int lane, const RotTurn& t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) turn[i] = lane + 32 * i < t.rot / 2 ? __ldg(t.turns + lane + 32 * i) : 0;
  }
  __device__ void fill(float* cs, int lane, int pos, const RotTurn& t) const {
    __syncwarp();  // the last token's have been read
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = lane + 32 * i;
      if (j < t.rot / 2) {
        const uint64_t a = static_cast<uint64_t>(turn[i]) * static_cast<uint64_t>(static_cast<int64_t>(pos));
        float s, c;
        sincospif(static_cast<float>(static_cast<int32_t>(a >> 32)) * 0x1p-31f, &s, &c);
        cs[j] = c * t.amp;
        cs[t.rot / 2 + j] = s * t.amp;
      }
    }
    __syncwarp();
  }
};

// A warp's part of the list, run by run: groups g0 .. g1 - 1 of token (row s of batch
// b), all of one kind (q, k or v).
struct RotWalk {
  int64_t left;
  int b, s, g0, g1, kind;
  bool token;  // the run is the token's first here
  __device__ RotWalk(const RotParams& p, int64_t i, int64_t n) : left(n), kind(0), token(true) {
    const int64_t row = i / p.first[3];
    g0 = g1 = static_cast<int>(i - row * p.first[3]);
    b = static_cast<int>(row / p.S);
    s = static_cast<int>(row - static_cast<int64_t>(b) * p.S);
    run(p);
  }
  __device__ void run(const RotParams& p) {
    kind = (g0 >= p.first[1]) + (g0 >= p.first[2]);
    const int end = kind == 0 ? p.first[1] : kind == 1 ? p.first[2] : p.first[3];
    g1 = static_cast<int>(min(static_cast<int64_t>(end), g0 + left));
  }
  __device__ bool next(const RotParams& p) {
    left -= g1 - g0;
    if (left <= 0) return false;
    g0 = g1;
    token = g0 == p.first[3];
    if (token) {
      g0 = 0;
      if (++s == p.S) s = 0, ++b;
    }
    run(p);
    return true;
  }
};
__device__ __forceinline__ uint16_t* rot_at(const RotRows& r, int b, int s, int head, int c0) {
  return r.p + b * r.b + s * r.row + head * r.head + c0;
}

// 8 packed channels as 4 pairs of fp32.
template <int kType>
__device__ __forceinline__ void rot_unpack(uint64_t* x, const uint4& w) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = unpack_16x2<kType>((&w.x)[e]);
    x[e] = pack_f32x2(f.x, f.y);
  }
}
template <int kType>
__device__ __forceinline__ uint4 rot_pack(const uint64_t* x) {
  uint4 w;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a, b;
    unpack_f32x2(x[e], a, b);
    (&w.x)[e] = pack_16x2<kType>(a, b);
  }
  return w;
}
// The words that hold the paired channels: another lane's, or this one's with their halves
// exchanged.  A channel that is not turned is paired with itself.
__device__ __forceinline__ uint4 rot_paired(const uint4& w, const RotTurn& t, int pair) {
  if (t.inter) return make_uint4(__byte_perm(w.x, 0u, pair), __byte_perm(w.y, 0u, pair), __byte_perm(w.z, 0u, pair),
                                 __byte_perm(w.w, 0u, pair));
  return make_uint4(__shfl_sync(0xffffffffu, w.x, pair), __shfl_sync(0xffffffffu, w.y, pair),
                    __shfl_sync(0xffffffffu, w.z, pair), __shfl_sync(0xffffffffu, w.w, pair));
}
__device__ __forceinline__ float rot_sum(uint64_t v) {
  float a, b;
  unpack_f32x2(v, a, b);
  return a + b;
}

// The weights of q and k (1 without a norm) as fp32, in shared memory.
template <int D, int kType>
__device__ __forceinline__ void rot_weights(float (*ws)[D], const RotParams& p) {
  for (int i = static_cast<int>(threadIdx.x); i < 2 * D; i += static_cast<int>(blockDim.x)) {
    const int kv = i / D, c = i % D;
    float w = 1.f;
    if (p.w[kv] != nullptr)
      w = p.w_fp32 ? __ldg(static_cast<const float*>(p.w[kv]) + c)
                   : unpack_16x2<kType>(__ldg(static_cast<const unsigned short*>(p.w[kv]) + c)).x;
    ws[kv][c] = w;
  }
}
__device__ __forceinline__ void rot_load8(float* x, const float* s) {
  const float4 a = *reinterpret_cast<const float4*>(s), b = *reinterpret_cast<const float4*>(s + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
// Cosines of this lane's channels, and sines with the sign that the paired channel has
// (forward; the gradient's is the other one).  A channel that is not turned is half of itself and
// half of itself again, which is itself: products with 0 would make NaN of an infinity.
template <int D>
__device__ __forceinline__ void rot_angles(float* co, float* si, const RotLane<D>& ln, const RotTurn& t, const float* cs) {
  if (!ln.turned) {
#pragma unroll
    for (int e = 0; e < 8; ++e) co[e] = 0.5f, si[e] = 0.5f;
  } else if (t.inter) {
    const float4 c = *reinterpret_cast<const float4*>(cs + ln.at), s = *reinterpret_cast<const float4*>(cs + t.rot / 2 + ln.at);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) co[e] = cc[e / 2], si[e] = e % 2 == 0 ? -ss[e / 2] : ss[e / 2];
  } else {
    rot_load8(co, cs + ln.at);
    rot_load8(si, cs + t.rot / 2 + ln.at);
    if (ln.low) {
#pragma unroll
      for (int e = 0; e < 8; ++e) si[e] = -si[e];
    }
  }
}

__device__ __forceinline__ uint4 rot_shared(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

struct NoPages {};

// Forward.  kPaged: tokens are packed rows, q goes to its rows and k and v to the
// pages (attn_paged.cuh says where).
template <int D, int kType, bool kPaged, typename Paged>
__device__ __forceinline__ void rot_forward_body(const RotParams& p, Paged pg) {
  using Lane = RotLane<D>;
  // Groups on their way.  16384 tokens of 64 heads took 92 / 89 / 92 / 97 / 98 us with 2 to
  // 6 (2 at four blocks an SM), 33021 tokens into pages of 16 138 / 139 / 132 / 134 with 3
  // to 6; in registers, four at once, 96 and 152.
  constexpr int kRing = kPaged ? 5 : 3;
  __shared__ __align__(16) uint4 ring_s[kRotWarps][kRing][32];
  __shared__ __align__(16) float cs_s[kRotWarps][D];
  __shared__ __align__(16) float w_s[2][D];
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const Lane ln(lane, p.turn);
  const uint32_t ring = smem_u32(&ring_s[warp][0][lane]);
  grid_dependency_wait();
  grid_launch_dependents();
  rot_weights<D, kType>(w_s, p);
  __syncthreads();
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * kRotWarps + warp) * p.share;
  if (i >= p.total) return;
  const RotTable table(lane, p.turn);
  float* const cs = cs_s[warp];
  RotWalk w(p, i, min(p.share, p.total - i));
  if constexpr (kPaged) pg.find(w.s);
  bool more = true;
  while (more) {
    const RotRows& in = p.in[w.kind];
    // this lane's head of the next group, and where its heads end
    int head = (w.g0 - p.first[w.kind]) * Lane::kRows + ln.sub, left = w.g1 - w.g0;
    const int end = min(p.heads[w.kind], (w.g1 - p.first[w.kind]) * Lane::kRows);
    const uint16_t* src = rot_at(in, w.b, w.s, head, ln.c0);
    const int64_t in_step = in.head * Lane::kRows;
    uint16_t* dst;
    int64_t out_step;
    bool keep = true;
    if constexpr (kPaged) {
      if (w.kind > 0) {
        keep = pg.to >= 0;
        out_step = pg.head_step * Lane::kRows;
        dst = (w.kind == 1 ? pg.k : pg.v) + (keep ? pg.to + head * pg.head_step + ln.c0 : 0);
      } else {
        keep = pg.live();
        out_step = p.out[0].head * Lane::kRows;
        dst = rot_at(p.out[0], 0, w.s, head, ln.c0);
      }
    } else {
      out_step = p.out[w.kind].head * Lane::kRows;
      dst = rot_at(p.out[w.kind], w.b, w.s, head, ln.c0);
    }
    const bool turns = !kPaged || w.kind < 2, norm = turns && p.w[w.kind & 1] != nullptr;
    uint64_t A[4], B[4];
    int ahead = head;
    const auto fetch = [&](int slot) {
      if (ahead < end) cp_async_16(ring + slot * 512, src);
      cp_async_commit();
      ahead += Lane::kRows;
      src += in_step;
    };
#pragma unroll
    for (int u = 0; u < kRing; ++u) fetch(u);
    if (turns) {  // while the first groups are on their way
      if (w.token && p.turn.rot > 0) {
        int pos;
        if constexpr (kPaged)
          pos = pg.pos;
        else
          pos = __ldg(p.pos + static_cast<int64_t>(w.b) * p.S + w.s);
        table.fill(cs, lane, pos, p.turn);
      }
      float co[8], si[8], own[8], other[8];
      rot_angles<D>(co, si, ln, p.turn, cs);
      rot_load8(own, w_s[w.kind & 1] + ln.c0);
      rot_load8(other, w_s[w.kind & 1] + (p.turn.inter ? ln.c0 : (ln.pair % Lane::kLanes) * 8));
      const bool swap = p.turn.inter && ln.turned;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float o0 = swap ? other[2 * e + 1] : other[2 * e], o1 = swap ? other[2 * e] : other[2 * e + 1];
        A[e] = pack_f32x2(co[2 * e] * own[2 * e], co[2 * e + 1] * own[2 * e + 1]);
        B[e] = pack_f32x2(si[2 * e] * o0, si[2 * e + 1] * o1);
      }
    }
    while (left > 0) {
#pragma unroll
      for (int u = 0; u < kRing; ++u) {
        if (left == 0) break;
        const bool there = head < end;
        cp_async_wait<kRing - 1>();  // this lane's copy of this group
        uint4 out = make_uint4(0, 0, 0, 0);
        if (there) out = rot_shared(ring + u * 512);
        if (turns) {
          uint64_t y[4], z[4];
          rot_unpack<kType>(y, out);
          rot_unpack<kType>(z, rot_paired(out, p.turn, ln.pair));
          fetch(u);
          float r = 1.f;
          if (norm) {
            uint64_t sq = mul_f32x2(y[0], y[0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) sq = fma_f32x2(y[e], y[e], sq);
            float ss = rot_sum(sq);
#pragma unroll
            for (int off = 1; off < Lane::kLanes; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            r = rsqrtf(fmaf(ss, 1.f / D, p.eps));
          }
          const uint64_t r2 = pack_f32x2(r, r);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = mul_f32x2(fma_f32x2(z[e], B[e], mul_f32x2(y[e], A[e])), r2);
          out = rot_pack<kType>(y);
        } else {
          fetch(u);
        }
        if (there && keep) *reinterpret_cast<uint4*>(dst) = out;
        head += Lane::kRows;
        dst += out_step;
        --left;
      }
    }
    cp_async_wait<0>();
    more = w.next(p);
    if constexpr (kPaged)
      if (more && w.token) pg.step(w.s);
  }
}

template <int D, int kType>
__global__ void __launch_bounds__(kRotThreads, kRotFwdBlocks) attn_norm_rope_kernel(const __grid_constant__ RotParams p) {
  rot_forward_body<D, kType, false>(p, NoPages{});
}

// Gradient, walked the same way.  A lane adds up g r x of its channels, for q and for
// k, in fp32 (its share's rows: 135 of 16384 tokens with 40 heads); the block's sums are added in
// shared memory, and a second kernel adds the blocks' in 64 bits: the same from call
// to call.
constexpr int kRotBwdThreads = 256;
constexpr int kRotBwdWarps = kRotBwdThreads / 32;
constexpr int kRotBwdBlocks = 2;  // blocks an SM

// A run of the gradient: heads of one kind; dw: its weight's sums.  dy and x come
// through the ring (in registers, four groups at once, it took 112 us instead of 108).
constexpr int kRotRing = 3;  // groups on their way (2 to 6: 111, 108, 109, 115, 119 us for 16384 tokens of 40 heads)
template <int D, int kType>
__device__ __forceinline__ void rot_backward_run(const RotParams& p, const RotWalk& w, const RotLane<D>& ln, const uint64_t* A,
                                                 const uint64_t* B, const float* w_s, uint64_t* dw, uint32_t ring) {
  using Lane = RotLane<D>;
  int head = (w.g0 - p.first[w.kind]) * Lane::kRows + ln.sub, left = w.g1 - w.g0, ahead = head;
  const int end = min(p.heads[w.kind], (w.g1 - p.first[w.kind]) * Lane::kRows);
  const bool norm = p.w[w.kind] != nullptr;
  const uint16_t* gsrc = rot_at(p.dy[w.kind], w.b, w.s, head, ln.c0);
  const uint16_t* xsrc = norm ? rot_at(p.in[w.kind], w.b, w.s, head, ln.c0) : gsrc;
  uint16_t* dst = rot_at(p.out[w.kind], w.b, w.s, head, ln.c0);
  const int64_t g_step = p.dy[w.kind].head * Lane::kRows, x_step = norm ? p.in[w.kind].head * Lane::kRows : 0,
                out_step = p.out[w.kind].head * Lane::kRows;
  const auto fetch = [&](int slot) {
    if (ahead < end) {
      cp_async_16(ring + slot * 1024, gsrc);
      if (norm) cp_async_16(ring + slot * 1024 + 512, xsrc);
    }
    cp_async_commit();
    ahead += Lane::kRows;
    gsrc += g_step;
    xsrc += x_step;
  };
#pragma unroll
  for (int u = 0; u < kRotRing; ++u) fetch(u);
  uint64_t wt[4];
  {
    float own[8];
    rot_load8(own, w_s + ln.c0);
#pragma unroll
    for (int e = 0; e < 4; ++e) wt[e] = pack_f32x2(own[2 * e], own[2 * e + 1]);
  }
  while (left > 0) {
#pragma unroll
    for (int u = 0; u < kRotRing; ++u) {
      if (left == 0) break;
      const bool there = head < end;
      cp_async_wait<kRotRing - 1>();  // this lane's copies of this group
      uint4 dy = make_uint4(0, 0, 0, 0), x = dy;
      if (there) {
        dy = rot_shared(ring + u * 1024);
        if (norm) x = rot_shared(ring + u * 1024 + 512);
      }
      uint64_t g[4], z[4];
      rot_unpack<kType>(g, dy);
      rot_unpack<kType>(z, rot_paired(dy, p.turn, ln.pair));
#pragma unroll
      for (int e = 0; e < 4; ++e) g[e] = fma_f32x2(z[e], B[e], mul_f32x2(g[e], A[e]));
      rot_unpack<kType>(z, x);
      fetch(u);
      if (norm) {
        uint64_t gw[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) gw[e] = mul_f32x2(g[e], wt[e]);
        uint64_t sq = mul_f32x2(z[0], z[0]), dt = mul_f32x2(gw[0], z[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) {
          sq = fma_f32x2(z[e], z[e], sq);
          dt = fma_f32x2(gw[e], z[e], dt);
        }
        float ss = rot_sum(sq), dot = rot_sum(dt);
#pragma unroll
        for (int off = 1; off < Lane::kLanes; off <<= 1) {
          ss += __shfl_xor_sync(0xffffffffu, ss, off);
          dot += __shfl_xor_sync(0xffffffffu, dot, off);
        }
        const float r = there ? rsqrtf(fmaf(ss, 1.f / D, p.eps)) : 0.f;  // (an eps of 0 is allowed)
        const float k = -r * r * dot * (1.f / D);
        const uint64_t r2 = pack_f32x2(r, r), k2 = pack_f32x2(k, k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dw[e] = fma_f32x2(g[e], mul_f32x2(r2, z[e]), dw[e]);
          g[e] = mul_f32x2(r2, fma_f32x2(k2, z[e], gw[e]));
        }
      }
      if (there) *reinterpret_cast<uint4*>(dst) = rot_pack<kType>(g);
      head += Lane::kRows;
      dst += out_step;
      --left;
    }
  }
  cp_async_wait<0>();
}

template <int D, int kType>
__global__ void __launch_bounds__(kRotBwdThreads, kRotBwdBlocks) attn_norm_rope_bwd_kernel(const __grid_constant__ RotParams p) {
  using Lane = RotLane<D>;
  __shared__ __align__(16) float cs_s[kRotBwdWarps][D];
  __shared__ __align__(16) float w_s[2][D];
  __shared__ __align__(16) uint4 ring_s[kRotBwdWarps][kRotRing][2][32];
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const Lane ln(lane, p.turn);
  const uint32_t ring = smem_u32(&ring_s[warp][0][0][lane]);
  grid_dependency_wait();
  grid_launch_dependents();
  rot_weights<D, kType>(w_s, p);
  __syncthreads();
  uint64_t dw[2][4];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[kv][e] = 0ull;
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * kRotBwdWarps + warp) * p.share;
  if (i < p.total) {
    const RotTable table(lane, p.turn);
    float* const cs = cs_s[warp];
    RotWalk w(p, i, min(p.share, p.total - i));
    uint64_t A[4], B[4];
    do {
      if (w.token) {
        if (p.turn.rot > 0) table.fill(cs, lane, __ldg(p.pos + static_cast<int64_t>(w.b) * p.S + w.s), p.turn);
        float co[8], si[8];
        rot_angles<D>(co, si, ln, p.turn, cs);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          A[e] = pack_f32x2(co[2 * e], co[2 * e + 1]);
          const float sign = ln.turned ? -1.f : 1.f;
          B[e] = pack_f32x2(sign * si[2 * e], sign * si[2 * e + 1]);
        }
      }
      if (w.kind == 0)
        rot_backward_run<D, kType>(p, w, ln, A, B, w_s[0], dw[0], ring);
      else
        rot_backward_run<D, kType>(p, w, ln, A, B, w_s[1], dw[1], ring);
    } while (w.next(p));
  }
  if (p.dw == nullptr) return;
  // the warp's rows, then the block's warps in their order
  float(*const part_s)[2][D] = reinterpret_cast<float(*)[2][D]>(ring_s);  // (no copy is under way any more)
  static_assert(sizeof(float) * kRotBwdWarps * 2 * D <= sizeof(ring_s), "the sums in the ring's room");
  __syncthreads();
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v[2];
      unpack_f32x2(dw[kv][e / 2], v[0], v[1]);
      float x = v[e % 2];
#pragma unroll
      for (int off = Lane::kLanes; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      if (ln.sub == 0) part_s[warp][kv][ln.c0 + e] = x;
    }
  __syncthreads();
  for (int j = tid; j < 2 * D; j += kRotBwdThreads) {
    float v = 0.f;
#pragma unroll
    for (int x = 0; x < kRotBwdWarps; ++x) v += part_s[x][j / D][j % D];
    p.dw[static_cast<int64_t>(blockIdx.x) * 2 * D + j] = v;
  }
}

// Sums of the blocks' weight gradients: 8 columns a block, a column's rows over 32
// threads.
constexpr int kRotSumThreads = 256;
template <int D>
__global__ void __launch_bounds__(kRotSumThreads) attn_norm_dw_kernel(const float* __restrict__ part, int blocks,
                                                                      float* __restrict__ dqw, float* __restrict__ dkw) {
  __shared__ double sum_s[kRotSumThreads / 32][8];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  const int col = static_cast<int>(blockIdx.x) * 8 + (tid & 7);
  grid_dependency_wait();
  grid_launch_dependents();
  double v = 0.0;
#pragma unroll 4
  for (int i = tid >> 3; i < blocks; i += kRotSumThreads / 8) v += static_cast<double>(__ldg(part + static_cast<int64_t>(i) * 2 * D + col));
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  v += __shfl_xor_sync(0xffffffffu, v, 16);
  if (lane < 8) sum_s[tid >> 5][lane] = v;
  __syncthreads();
  if (tid < 8) {
    v = 0.0;
#pragma unroll
    for (int i = 0; i < kRotSumThreads / 32; ++i) v += sum_s[i][tid];
    float* const out = col < D ? dqw : dkw;
    if (out != nullptr) out[col % D] = static_cast<float>(v);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Shares of a pass: one a warp, at most as many warps as the SMs hold at once.
struct RotGrid {
  int64_t total, share;
  unsigned blocks;
};
RotGrid rot_grid(int64_t tokens, int groups, int sms, int blocks_per_sm, int warps_per_block) {
  RotGrid g;
  g.total = tokens * groups;
  const int64_t warps = static_cast<int64_t>(sms) * blocks_per_sm * warps_per_block;
  g.share = (g.total + warps - 1) / warps;
  const int64_t used = g.share > 0 ? (g.total + g.share - 1) / g.share : 0;
  g.blocks = static_cast<unsigned>((used + warps_per_block - 1) / warps_per_block);
  return g;
}

bool rot_rows_ok(const attn_heads_t* r, attn_status_t* st) {
  *st = r == nullptr || r->ptr == nullptr ? ATTN_ERR_INVALID_ARG
        : !aligned(r->ptr, 16) || r->batch_stride % 8 != 0 || r->row_stride % 8 != 0 || r->head_stride % 8 != 0
            ? ATTN_ERR_ALIGNMENT
            : ATTN_OK;
  return *st == ATTN_OK;
}
RotRows rot_rows_of(const attn_heads_t* r) {
  return {static_cast<uint16_t*>(r->ptr), r->batch_stride, r->row_stride, r->head_stride};
}

attn_status_t rot_check_turn(const attn_rotary_t* t, int D, RotTurn* out) {
  *out = RotTurn{nullptr, 0, 0, 1.f};
  if (t == nullptr) return ATTN_OK;
  if (t->rot < 0 || t->rot > D || (t->interleaved != 0 && t->interleaved != 1) || !std::isfinite(t->amplitude))
    return ATTN_ERR_INVALID_ARG;
  if (t->rot > 0 && t->turns == nullptr) return ATTN_ERR_INVALID_ARG;
  if (t->rot % 16 != 0) return ATTN_ERR_UNSUPPORTED;
  if (!aligned(t->turns, 8)) return ATTN_ERR_ALIGNMENT;
  *out = RotTurn{t->turns, t->rot, t->interleaved, t->amplitude};
  return ATTN_OK;
}
// Weights of both or of one, and what goes with them.
attn_status_t rot_check_norm(const void* qw, const void* kw, int w_dtype, int dtype, float eps) {
  if (qw == nullptr && kw == nullptr) return ATTN_OK;
  if (w_dtype != dtype && w_dtype != ATTN_FP32) return ATTN_ERR_UNSUPPORTED;
  if (!std::isfinite(eps) || eps < 0.f) return ATTN_ERR_INVALID_ARG;
  const uintptr_t a = w_dtype == ATTN_FP32 ? 4 : 2;
  return aligned(qw, a) && aligned(kw, a) ? ATTN_OK : ATTN_ERR_ALIGNMENT;
}

// Heads of q, k and v, and their groups in a token's list; returns the groups.
int rot_groups(RotParams* p, int D, int H_q, int H_k, int H_v) {
  const int h[3] = {H_q, H_k, H_v}, rows = 32 / (D / 8);
  p->first[0] = 0;
  for (int i = 0; i < 3; ++i) {
    p->heads[i] = h[i];
    p->first[i + 1] = p->first[i] + (h[i] + rows - 1) / rows;
  }
  return p->first[3];
}

attn_status_t rot_check_shape(int B, int S, int H_q, int H_k, int D, int dtype) {
  if (B < 0 || S < 0 || H_q < 1 || H_k < 1) return ATTN_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || (dtype != ATTN_BF16 && dtype != ATTN_FP16) || H_q > 65535 || H_k > 65535 ||
      static_cast<int64_t>(B) * S > INT_MAX)
    return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// (SMs of a GB300: the workspace's size is asked for without a device)
constexpr int kRotSms = 152;

}  // namespace

extern "C" {

attn_status_t attn_qk_norm_rope(const attn_heads_t* q, const attn_heads_t* k, const attn_heads_t* q_out,
                                const attn_heads_t* k_out, int B, int S, int H_q, int H_k, int D, int dtype,
                                const attn_rotary_t* rope, const int32_t* positions, const void* q_weight,
                                const void* k_weight, int weight_dtype, float eps, void* stream) {
  attn_status_t st = rot_check_shape(B, S, H_q, H_k, D, dtype);
  if (st != ATTN_OK) return st;
  RotParams p{};
  st = rot_check_turn(rope, D, &p.turn);
  if (st != ATTN_OK) return st;
  st = rot_check_norm(q_weight, k_weight, weight_dtype, dtype, eps);
  if (st != ATTN_OK) return st;
  if (B == 0 || S == 0) return ATTN_OK;
  if (p.turn.rot > 0 && positions == nullptr) return ATTN_ERR_INVALID_ARG;
  if (!rot_rows_ok(q, &st) || !rot_rows_ok(k, &st) || !rot_rows_ok(q_out, &st) || !rot_rows_ok(k_out, &st)) return st;
  if (!aligned(positions, 4)) return ATTN_ERR_ALIGNMENT;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_DEVICE;
  st = prepare_device(dev);
  if (st != ATTN_OK) return st;
  p.in[0] = rot_rows_of(q), p.in[1] = rot_rows_of(k);
  p.out[0] = rot_rows_of(q_out), p.out[1] = rot_rows_of(k_out);
  p.w[0] = q_weight, p.w[1] = k_weight;
  p.w_fp32 = weight_dtype == ATTN_FP32;
  p.eps = eps;
  p.pos = positions;
  p.S = S;
  const RotGrid g = rot_grid(static_cast<int64_t>(B) * S, rot_groups(&p, D, H_q, H_k, 0),
                             g_dev_sms[dev].load(std::memory_order_relaxed), kRotFwdBlocks, kRotWarps);
  p.total = g.total, p.share = g.share;
  const auto run = [&](auto kernel) {
    return launch_pdl(kernel, dim3(g.blocks), dim3(kRotThreads), 0, static_cast<cudaStream_t>(stream), p);
  };
  const bool bf = dtype == ATTN_BF16;
  const cudaError_t e = D == 64 ? (bf ? run(attn_norm_rope_kernel<64, kBF16>) : run(attn_norm_rope_kernel<64, kFP16>))
                                : (bf ? run(attn_norm_rope_kernel<128, kBF16>) : run(attn_norm_rope_kernel<128, kFP16>));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

uint64_t attn_qk_norm_rope_bwd_workspace_bytes(int B, int S, int H_q, int H_k, int D) {
  if (rot_check_shape(B, S, H_q, H_k, D, ATTN_BF16) != ATTN_OK) return 0;
  if (B == 0 || S == 0) return 16;
  RotParams p{};
  return static_cast<uint64_t>(rot_grid(static_cast<int64_t>(B) * S, rot_groups(&p, D, H_q, H_k, 0), kRotSms, kRotBwdBlocks, kRotBwdWarps).blocks) * 2 *
         D * sizeof(float);
}

attn_status_t attn_qk_norm_rope_bwd(const attn_heads_t* dq_out, const attn_heads_t* dk_out, const attn_heads_t* q,
                                    const attn_heads_t* k, const attn_heads_t* dq, const attn_heads_t* dk, int B, int S,
                                    int H_q, int H_k, int D, int dtype, const attn_rotary_t* rope, const int32_t* positions,
                                    const void* q_weight, const void* k_weight, int weight_dtype, float eps,
                                    float* dq_weight, float* dk_weight, void* workspace, uint64_t workspace_bytes,
                                    void* stream) {
  attn_status_t st = rot_check_shape(B, S, H_q, H_k, D, dtype);
  if (st != ATTN_OK) return st;
  RotParams p{};
  st = rot_check_turn(rope, D, &p.turn);
  if (st != ATTN_OK) return st;
  st = rot_check_norm(q_weight, k_weight, weight_dtype, dtype, eps);
  if (st != ATTN_OK) return st;
  if ((q_weight != nullptr) != (dq_weight != nullptr) || (k_weight != nullptr) != (dk_weight != nullptr)) return ATTN_ERR_INVALID_ARG;
  const bool norm = q_weight != nullptr || k_weight != nullptr, rows = B > 0 && S > 0;
  if (rows) {
    if (p.turn.rot > 0 && positions == nullptr) return ATTN_ERR_INVALID_ARG;
    if (!rot_rows_ok(dq_out, &st) || !rot_rows_ok(dk_out, &st) || !rot_rows_ok(dq, &st) || !rot_rows_ok(dk, &st)) return st;
    if ((q_weight != nullptr && !rot_rows_ok(q, &st)) || (k_weight != nullptr && !rot_rows_ok(k, &st))) return st;
  }
  if (!aligned(positions, 4) || !aligned(dq_weight, 4) || !aligned(dk_weight, 4) || !aligned(workspace, 16)) return ATTN_ERR_ALIGNMENT;
  if (norm && (workspace == nullptr || workspace_bytes < attn_qk_norm_rope_bwd_workspace_bytes(B, S, H_q, H_k, D))) return ATTN_ERR_INVALID_ARG;
  if (!rows && !norm) return ATTN_OK;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_DEVICE;
  st = prepare_device(dev);
  if (st != ATTN_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  unsigned blocks = 0;
  if (rows) {
    p.dy[0] = rot_rows_of(dq_out), p.dy[1] = rot_rows_of(dk_out);
    if (q_weight != nullptr) p.in[0] = rot_rows_of(q);
    if (k_weight != nullptr) p.in[1] = rot_rows_of(k);
    p.out[0] = rot_rows_of(dq), p.out[1] = rot_rows_of(dk);
    p.w[0] = q_weight, p.w[1] = k_weight;
    p.w_fp32 = weight_dtype == ATTN_FP32;
    p.eps = eps;
    p.pos = positions;
    p.S = S;
    // (the grid is a GB300's whatever the device has: it sizes the workspace)
    const RotGrid g = rot_grid(static_cast<int64_t>(B) * S, rot_groups(&p, D, H_q, H_k, 0), kRotSms, kRotBwdBlocks, kRotBwdWarps);
    p.total = g.total, p.share = g.share;
    p.dw = norm ? static_cast<float*>(workspace) : nullptr;
    blocks = g.blocks;
    const auto run = [&](auto kernel) { return launch_pdl(kernel, dim3(g.blocks), dim3(kRotBwdThreads), 0, s, p); };
    const bool bf = dtype == ATTN_BF16;
    e = D == 64 ? (bf ? run(attn_norm_rope_bwd_kernel<64, kBF16>) : run(attn_norm_rope_bwd_kernel<64, kFP16>))
                : (bf ? run(attn_norm_rope_bwd_kernel<128, kBF16>) : run(attn_norm_rope_bwd_kernel<128, kFP16>));
  }
  if (e == cudaSuccess && norm) {
    const auto run = [&](auto kernel) {
      return launch_pdl(kernel, dim3(static_cast<unsigned>(2 * D / 8)), dim3(kRotSumThreads), 0, s, static_cast<const float*>(workspace),
                        static_cast<int>(blocks), dq_weight, dk_weight);
    };
    e = D == 64 ? run(attn_norm_dw_kernel<64>) : run(attn_norm_dw_kernel<128>);
  }
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

}  // extern "C"
