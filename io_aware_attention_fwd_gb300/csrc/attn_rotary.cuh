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
// A row of 256 (128) bytes is 16 (8) lanes of 8 channels; what pairs with them is
// one shuffle of the 16-bit words away.  A block takes up to 8 tokens: their
// cosines and sines are worked out once, in shared memory, for all heads.

namespace {

constexpr int kRotThreads = 256;
constexpr int kRotWarps = kRotThreads / 32;
constexpr int kRotTokens = 8;  // tokens a block takes at once, at most

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
  int groups[3];   // of the heads a warp takes at once
  const void* w[2];  // weights, or null: no norm
  int w_fp32;
  float eps;
  RotTurn turn;
  const int32_t* pos;  // [B][S]
  int B, S;
  int tokens;      // a block's
  int tiles;       // ceil(S / tokens)
  int per_block;   // groups a block takes (its blockIdx.y-th part of them)
  float* dw;       // gradient: [blocks][2][D]
};

// What the lanes of a row hold.
template <int D>
struct RotLane {
  static constexpr int kLanes = D / 8;          // lanes a row
  static constexpr int kRows = 32 / kLanes;     // rows a warp
  int sub, c0;                                  // this lane's row of the warp's, and first channel
  int partner;                                  // lane with the paired channels (half layout)
  float sign;                                   // of the paired channel's sine
  bool turned;
  int at;                                       // of its first cosine
  __device__ RotLane(int lane, const RotTurn& t) {
    sub = lane / kLanes;
    c0 = (lane % kLanes) * 8;
    const int half = t.rot / 2;
    turned = c0 < t.rot;
    const bool low = c0 < half;
    partner = t.inter || !turned ? lane : lane + (low ? half : -half) / 8;
    sign = low ? -1.f : 1.f;
    at = t.inter ? c0 / 2 : low ? c0 : c0 - half;
  }
};

// Cosines and sines of a block's tokens: cs[token][0 .. rot/2 - 1] and the sines behind.
__device__ __forceinline__ void rot_table(float* cs, const int* pos, int tokens, const RotTurn& t) {
  const int half = t.rot / 2;
  for (int i = static_cast<int>(threadIdx.x); i < tokens * half; i += kRotThreads) {
    const int tok = i / half, j = i - tok * half;
    const uint64_t turn = static_cast<uint64_t>(__ldg(t.turns + j)) * static_cast<uint64_t>(static_cast<int64_t>(pos[tok]));
    const int32_t half_turns = static_cast<int32_t>(turn >> 32);
    float s, c;
    sincospif(static_cast<float>(half_turns) * 0x1p-31f, &s, &c);
    cs[tok * t.rot + j] = c * t.amp;
    cs[tok * t.rot + half + j] = s * t.amp;
  }
}

template <int kType>
__device__ __forceinline__ void rot_unpack(float* x, const uint4& w) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = unpack_16x2<kType>((&w.x)[e]);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
}
template <int kType>
__device__ __forceinline__ uint4 rot_pack(const float* x) {
  return make_uint4(pack_16x2<kType>(x[0], x[1]), pack_16x2<kType>(x[2], x[3]), pack_16x2<kType>(x[4], x[5]),
                    pack_16x2<kType>(x[6], x[7]));
}
__device__ __forceinline__ uint4 rot_shuffle(const uint4& w, int from) {
  return make_uint4(__shfl_sync(0xffffffffu, w.x, from), __shfl_sync(0xffffffffu, w.y, from),
                    __shfl_sync(0xffffffffu, w.z, from), __shfl_sync(0xffffffffu, w.w, from));
}
__device__ __forceinline__ void rot_load8(float* x, const float* s) {
  const float4 a = *reinterpret_cast<const float4*>(s), b = *reinterpret_cast<const float4*>(s + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// Turns x (this lane's 8 channels) by the token's angles, backwards if kBack; y
// holds the paired channels in the half layout.
template <bool kBack>
__device__ __forceinline__ void rot_turn(float* x, const float* y, const float* cs, const RotTurn& t, float sign, int at) {
  if (t.inter) {
    const float4 c = *reinterpret_cast<const float4*>(cs + at), s = *reinterpret_cast<const float4*>(cs + t.rot / 2 + at);
    const float co[4] = {c.x, c.y, c.z, c.w}, si[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = x[2 * e], b = x[2 * e + 1], sn = kBack ? -si[e] : si[e];
      x[2 * e] = fmaf(a, co[e], -b * sn);
      x[2 * e + 1] = fmaf(a, sn, b * co[e]);
    }
  } else {
    float co[8], si[8];
    rot_load8(co, cs + at);
    rot_load8(si, cs + t.rot / 2 + at);
    if (kBack) sign = -sign;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], co[e], sign * y[e] * si[e]);
  }
}

// The weights of q and k as fp32, in shared memory.
template <int D, int kType>
__device__ __forceinline__ void rot_weights(float (*ws)[D], const RotParams& p) {
  for (int i = static_cast<int>(threadIdx.x); i < 2 * D; i += kRotThreads) {
    const int kv = i / D, c = i % D;
    float w = 1.f;
    if (p.w[kv] != nullptr) {
      if (p.w_fp32) {
        w = __ldg(static_cast<const float*>(p.w[kv]) + c);
      } else {
        const float2 f = unpack_16x2<kType>(__ldg(static_cast<const unsigned short*>(p.w[kv]) + c));
        w = f.x;
      }
    }
    ws[kv][c] = w;
  }
}

// One group of heads of one token, as a warp takes them.
struct RotItem {
  int tok, kind, head;
  bool there;
};
template <int D>
__device__ __forceinline__ RotItem rot_item(const RotParams& p, int tok, int group, int sub, int tokens) {
  RotItem it{tok, 0, 0, false};
  if (tok >= tokens) return it;
  if (group >= p.groups[0]) group -= p.groups[0], it.kind = 1;
  if (it.kind == 1 && group >= p.groups[1]) group -= p.groups[1], it.kind = 2;
  it.head = group * RotLane<D>::kRows + sub;
  it.there = it.head < p.heads[it.kind];
  return it;
}

template <int D, int kType>
__device__ __forceinline__ uint4 rot_load(const RotRows& r, int64_t at) {
  return *reinterpret_cast<const uint4*>(r.p + at);
}

// x normed (w: this lane's weights and, half layout, its partners') and turned.
template <int D, int kType>
__device__ __forceinline__ uint4 rot_forward(const uint4& raw, const float* w, const float* cs, const RotParams& p, bool norm,
                                             const RotLane<D>& ln, int partner_c0) {
  float x[8], y[8];
  rot_unpack<kType>(x, raw);
  float r = 1.f;
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int off = 1; off < RotLane<D>::kLanes; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    r = rsqrtf(fmaf(ss, 1.f / D, p.eps));
  }
  if (!p.turn.inter && p.turn.rot > 0) rot_unpack<kType>(y, rot_shuffle(raw, ln.partner));
  if (norm) {
    float ww[8];
    rot_load8(ww, w + ln.c0);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= r * ww[e];
    if (!p.turn.inter && p.turn.rot > 0) {
      rot_load8(ww, w + partner_c0);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= r * ww[e];
    }
  }
  if (ln.turned) rot_turn<false>(x, y, cs, p.turn, ln.sign, ln.at);
  return rot_pack<kType>(x);
}

// Forward.  kPaged: tokens are packed rows, q goes to its rows and k and v to
// the pages (attn_paged.cuh says where: paged_place).
template <int D, int kType, bool kPaged, typename Paged>
__device__ __forceinline__ void rot_forward_body(const RotParams& p, const Paged& pg) {
  using Lane = RotLane<D>;
  constexpr int kBatch = 4;  // rows a lane has in flight
  __shared__ __align__(16) float cs_s[kRotTokens * D];
  __shared__ __align__(16) float w_s[2][D];
  __shared__ int pos_s[kRotTokens];
  __shared__ int64_t to_s[kRotTokens];  // kPaged: first element of the token's row in its page; -1: in none
  __shared__ int live_s[kRotTokens];    // kPaged: the row belongs to a sequence
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const Lane ln(lane, p.turn);
  const int partner_c0 = (ln.partner % Lane::kLanes) * 8;
  const int b = static_cast<int>(blockIdx.x) / p.tiles, tile = static_cast<int>(blockIdx.x) - b * p.tiles;
  const int s0 = tile * p.tokens, tokens = min(p.tokens, p.S - s0);
  const int g0 = static_cast<int>(blockIdx.y) * p.per_block;
  const int all = p.groups[0] + p.groups[1] + (kPaged ? p.groups[2] : 0);
  const int ng = min(p.per_block, all - g0);
  grid_dependency_wait();
  grid_launch_dependents();

  int tok = 0, g = warp;  // this warp's next item
  while (g >= ng && tok < tokens) g -= ng, ++tok;
  uint4 raw[kBatch];
  RotItem it[kBatch];
  const auto fetch = [&]() {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      it[u] = rot_item<D>(p, tok, g0 + g, ln.sub, tokens);
      raw[u] = make_uint4(0, 0, 0, 0);
      if (it[u].there) {
        const RotRows& r = p.in[it[u].kind];
        raw[u] = rot_load<D, kType>(r, b * r.b + (s0 + tok) * r.row + it[u].head * r.head + ln.c0);
      }
      g += kRotWarps;
      while (g >= ng && tok < tokens) g -= ng, ++tok;
    }
  };
  fetch();  // on their way while the angles are worked out
  if (tid < tokens) {
    if constexpr (kPaged) {
      int pos, live;
      to_s[tid] = pg.template place<D>(s0 + tid, &pos, &live, blockIdx.y == 0);
      pos_s[tid] = pos;
      live_s[tid] = live;
    } else {
      pos_s[tid] = p.pos != nullptr ? __ldg(p.pos + static_cast<int64_t>(b) * p.S + s0 + tid) : 0;
    }
  }
  rot_weights<D, kType>(w_s, p);
  __syncthreads();
  rot_table(cs_s, pos_s, tokens, p.turn);
  __syncthreads();
  while (it[0].tok < tokens) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int t = min(it[u].tok, tokens - 1), kind = it[u].kind;
      uint4 y = raw[u];
      if (!kPaged || kind < 2)  // (the whole warp: an item is of one kind)
        y = rot_forward<D, kType>(raw[u], w_s[kind & 1], cs_s + t * p.turn.rot, p, p.w[kind & 1] != nullptr, ln, partner_c0);
      if (!it[u].there) continue;
      if (kPaged && kind > 0) {
        const int64_t to = to_s[t];
        if (to >= 0)
          *reinterpret_cast<uint4*>((kind == 1 ? pg.k : pg.v) + to + static_cast<int64_t>(it[u].head) * pg.head_step + ln.c0) = y;
      } else if (!kPaged || live_s[t]) {
        const RotRows& r = p.out[kind];
        *reinterpret_cast<uint4*>(r.p + b * r.b + (s0 + t) * r.row + it[u].head * r.head + ln.c0) = y;
      }
    }
    fetch();
  }
}

struct NoPages {
  uint16_t *k, *v;
  int64_t head_step;
};
template <int D, int kType>
__global__ void __launch_bounds__(kRotThreads) attn_norm_rope_kernel(const __grid_constant__ RotParams p) {
  rot_forward_body<D, kType, false>(p, NoPages{});
}

// Gradient.  A block walks tiles of tokens; its lanes add up g r x of their
// channels, for q and for k, in fp32 (some hundred rows each), the block's sums
// are added in shared memory, and a second kernel adds the blocks' in 64 bits:
// the same from call to call.
template <int D, int kType>
__global__ void __launch_bounds__(kRotThreads) attn_norm_rope_bwd_kernel(const __grid_constant__ RotParams p) {
  using Lane = RotLane<D>;
  constexpr int kBatch = 2;
  __shared__ __align__(16) float cs_s[kRotTokens * D];
  __shared__ __align__(16) float w_s[2][D];
  __shared__ int pos_s[kRotTokens];
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const Lane ln(lane, p.turn);
  const int g0 = static_cast<int>(blockIdx.y) * p.per_block;
  const int ng = min(p.per_block, p.groups[0] + p.groups[1] - g0);
  grid_dependency_wait();
  grid_launch_dependents();
  rot_weights<D, kType>(w_s, p);
  float dw[2][8];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[kv][e] = 0.f;
  const int n_tiles = p.B * p.tiles;
  for (int x = static_cast<int>(blockIdx.x); x < n_tiles; x += static_cast<int>(gridDim.x)) {
    const int b = x / p.tiles, tile = x - b * p.tiles;
    const int s0 = tile * p.tokens, tokens = min(p.tokens, p.S - s0);
    int tok = 0, g = warp;
    while (g >= ng && tok < tokens) g -= ng, ++tok;
    uint4 raw[kBatch], draw[kBatch];
    RotItem it[kBatch];
    const auto fetch = [&]() {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        it[u] = rot_item<D>(p, tok, g0 + g, ln.sub, tokens);
        raw[u] = draw[u] = make_uint4(0, 0, 0, 0);
        if (it[u].there) {
          const int kind = it[u].kind;
          const RotRows& r = p.dy[kind];
          draw[u] = rot_load<D, kType>(r, b * r.b + (s0 + tok) * r.row + it[u].head * r.head + ln.c0);
          if (p.w[kind] != nullptr) {
            const RotRows& q = p.in[kind];
            raw[u] = rot_load<D, kType>(q, b * q.b + (s0 + tok) * q.row + it[u].head * q.head + ln.c0);
          }
        }
        g += kRotWarps;
        while (g >= ng && tok < tokens) g -= ng, ++tok;
      }
    };
    fetch();
    __syncthreads();  // the last tile's angles have been used
    if (tid < tokens) pos_s[tid] = p.pos != nullptr ? __ldg(p.pos + static_cast<int64_t>(b) * p.S + s0 + tid) : 0;
    __syncthreads();
    rot_table(cs_s, pos_s, tokens, p.turn);
    __syncthreads();
    while (it[0].tok < tokens) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int t = min(it[u].tok, tokens - 1), kind = it[u].kind;
        float gr[8], y[8];
        rot_unpack<kType>(gr, draw[u]);
        if (!p.turn.inter && p.turn.rot > 0) rot_unpack<kType>(y, rot_shuffle(draw[u], ln.partner));
        if (ln.turned) rot_turn<true>(gr, y, cs_s + t * p.turn.rot, p.turn, ln.sign, ln.at);
        if (p.w[kind] != nullptr) {
          float xv[8], ww[8];
          rot_unpack<kType>(xv, raw[u]);
          rot_load8(ww, w_s[kind] + ln.c0);
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ss = fmaf(xv[e], xv[e], ss);
            ww[e] *= gr[e];
            dot = fmaf(ww[e], xv[e], dot);
          }
#pragma unroll
          for (int off = 1; off < Lane::kLanes; off <<= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, off);
            dot += __shfl_xor_sync(0xffffffffu, dot, off);
          }
          const float r = it[u].there ? rsqrtf(fmaf(ss, 1.f / D, p.eps)) : 0.f;  // (an eps of 0 is allowed)
          const float k = r * r * dot * (1.f / D);
          if (kind == 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) dw[0][e] = fmaf(gr[e], r * xv[e], dw[0][e]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) dw[1][e] = fmaf(gr[e], r * xv[e], dw[1][e]);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) gr[e] = r * fmaf(-k, xv[e], ww[e]);
        }
        if (!it[u].there) continue;
        const RotRows& o = p.out[kind];
        *reinterpret_cast<uint4*>(o.p + b * o.b + (s0 + t) * o.row + it[u].head * o.head + ln.c0) = rot_pack<kType>(gr);
      }
      fetch();
    }
  }
  if (p.dw == nullptr) return;
  // the warp's rows, then the block's warps in their order
  __shared__ float part_s[kRotWarps][2][D];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v = dw[kv][e];
#pragma unroll
      for (int off = Lane::kLanes; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
      if (ln.sub == 0) part_s[warp][kv][ln.c0 + e] = v;
    }
  __syncthreads();
  const int64_t block = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
  for (int i = tid; i < 2 * D; i += kRotThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kRotWarps; ++w) v += part_s[w][i / D][i % D];
    p.dw[block * 2 * D + i] = v;
  }
}

// Sums of the blocks' weight gradients: 32 columns a block, a column's rows over
// 32 threads.
template <int D>
__global__ void __launch_bounds__(1024) attn_norm_dw_kernel(const float* __restrict__ part, int blocks, float* __restrict__ dqw,
                                                            float* __restrict__ dkw) {
  __shared__ double sum_s[32][33];
  const int cx = static_cast<int>(threadIdx.x) & 31, y = static_cast<int>(threadIdx.x) >> 5;
  const int col = static_cast<int>(blockIdx.x) * 32 + cx;
  grid_dependency_wait();
  grid_launch_dependents();
  double v = 0.0;
  for (int i = y; i < blocks; i += 32) v += static_cast<double>(__ldg(part + static_cast<int64_t>(i) * 2 * D + col));
  sum_s[y][cx] = v;
  __syncthreads();
  if (y == 0) {
    for (int i = 1; i < 32; ++i) v += sum_s[i][cx];
    float* const out = col < D ? dqw : dkw;
    if (out != nullptr) out[col % D] = static_cast<float>(v);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Blocks of a pass over rows [B][S]: tokens a block, and parts of the heads
// (more of both for few rows, so that they fill the SMs: two blocks each).
struct RotGrid {
  int tokens, tiles, per_block;
  unsigned parts;
  int64_t blocks;  // B * tiles
};
RotGrid rot_grid(int B, int S, int groups, int sms) {
  RotGrid g;
  g.tokens = std::min(kRotTokens, S);
  const auto count = [&](int t) { return static_cast<int64_t>(B) * ((S + t - 1) / t); };
  while (g.tokens > 1 && count(g.tokens) < 2 * sms) g.tokens /= 2;
  g.blocks = count(g.tokens);
  g.tiles = (S + g.tokens - 1) / g.tokens;
  g.parts = 1;
  if (g.blocks < 2 * sms) g.parts = static_cast<unsigned>((groups + kRotWarps - 1) / kRotWarps);
  g.per_block = (groups + static_cast<int>(g.parts) - 1) / static_cast<int>(g.parts);
  g.parts = static_cast<unsigned>((groups + g.per_block - 1) / g.per_block);
  return g;
}

constexpr int kRotBwdBlocks = 4;  // blocks an SM that walk the tiles

bool rot_rows_ok(const attn_heads_t* r, int D, attn_status_t* st) {
  *st = r == nullptr || r->ptr == nullptr ? ATTN_ERR_INVALID_ARG
        : !aligned(r->ptr, 16) || r->batch_stride % 8 != 0 || r->row_stride % 8 != 0 || r->head_stride % 8 != 0
            ? ATTN_ERR_ALIGNMENT
            : ATTN_OK;
  (void)D;
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

template <int D>
void rot_groups(RotParams* p, int H_q, int H_k, int H_v) {
  const int h[3] = {H_q, H_k, H_v};
  for (int i = 0; i < 3; ++i) {
    p->heads[i] = h[i];
    p->groups[i] = (h[i] + RotLane<D>::kRows - 1) / RotLane<D>::kRows;
  }
}
void rot_groups(RotParams* p, int D, int H_q, int H_k, int H_v) {
  if (D == 64)
    rot_groups<64>(p, H_q, H_k, H_v);
  else
    rot_groups<128>(p, H_q, H_k, H_v);
}

attn_status_t rot_check_shape(int B, int S, int H_q, int H_k, int D, int dtype) {
  if (B < 0 || S < 0 || H_q < 1 || H_k < 1) return ATTN_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || (dtype != ATTN_BF16 && dtype != ATTN_FP16) || H_q > 65535 || H_k > 65535 ||
      static_cast<int64_t>(B) * S > INT_MAX)
    return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

int64_t rot_bwd_blocks(const RotGrid& g, int sms) { return std::min<int64_t>(g.blocks, static_cast<int64_t>(kRotBwdBlocks) * sms); }

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
  if (!rot_rows_ok(q, D, &st) || !rot_rows_ok(k, D, &st) || !rot_rows_ok(q_out, D, &st) || !rot_rows_ok(k_out, D, &st)) return st;
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
  p.B = B, p.S = S;
  rot_groups(&p, D, H_q, H_k, 0);
  const RotGrid g = rot_grid(B, S, p.groups[0] + p.groups[1], g_dev_sms[dev].load(std::memory_order_relaxed));
  p.tokens = g.tokens, p.tiles = g.tiles, p.per_block = g.per_block;
  const auto run = [&](auto kernel) {
    return launch_pdl(kernel, dim3(static_cast<unsigned>(g.blocks), g.parts), dim3(kRotThreads), 0,
                      static_cast<cudaStream_t>(stream), p);
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
  rot_groups(&p, D, H_q, H_k, 0);
  const RotGrid g = rot_grid(B, S, p.groups[0] + p.groups[1], kRotSms);
  return static_cast<uint64_t>(rot_bwd_blocks(g, kRotSms)) * g.parts * 2 * D * sizeof(float);
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
    if (!rot_rows_ok(dq_out, D, &st) || !rot_rows_ok(dk_out, D, &st) || !rot_rows_ok(dq, D, &st) || !rot_rows_ok(dk, D, &st)) return st;
    if ((q_weight != nullptr && !rot_rows_ok(q, D, &st)) || (k_weight != nullptr && !rot_rows_ok(k, D, &st))) return st;
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
  int64_t blocks = 0;
  if (rows) {
    p.dy[0] = rot_rows_of(dq_out), p.dy[1] = rot_rows_of(dk_out);
    if (q_weight != nullptr) p.in[0] = rot_rows_of(q);
    if (k_weight != nullptr) p.in[1] = rot_rows_of(k);
    p.out[0] = rot_rows_of(dq), p.out[1] = rot_rows_of(dk);
    p.w[0] = q_weight, p.w[1] = k_weight;
    p.w_fp32 = weight_dtype == ATTN_FP32;
    p.eps = eps;
    p.pos = positions;
    p.B = B, p.S = S;
    rot_groups(&p, D, H_q, H_k, 0);
    // (the grid is a GB300's whatever the device has: it sizes the workspace)
    const RotGrid g = rot_grid(B, S, p.groups[0] + p.groups[1], kRotSms);
    p.tokens = g.tokens, p.tiles = g.tiles, p.per_block = g.per_block;
    p.dw = norm ? static_cast<float*>(workspace) : nullptr;
    const int64_t gx = rot_bwd_blocks(g, kRotSms);
    blocks = gx * g.parts;
    const auto run = [&](auto kernel) {
      return launch_pdl(kernel, dim3(static_cast<unsigned>(gx), g.parts), dim3(kRotThreads), 0, s, p);
    };
    const bool bf = dtype == ATTN_BF16;
    e = D == 64 ? (bf ? run(attn_norm_rope_bwd_kernel<64, kBF16>) : run(attn_norm_rope_bwd_kernel<64, kFP16>))
                : (bf ? run(attn_norm_rope_bwd_kernel<128, kBF16>) : run(attn_norm_rope_bwd_kernel<128, kFP16>));
  }
  if (e == cudaSuccess && norm) {
    const auto run = [&](auto kernel) {
      return launch_pdl(kernel, dim3(static_cast<unsigned>(2 * D / 32)), dim3(1024), 0, s, static_cast<const float*>(workspace),
                        static_cast<int>(blocks), dq_weight, dk_weight);
    };
    e = D == 64 ? run(attn_norm_dw_kernel<64>) : run(attn_norm_dw_kernel<128>);
  }
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

}  // extern "C"
