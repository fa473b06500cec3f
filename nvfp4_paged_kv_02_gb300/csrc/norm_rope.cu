// norm_rope.cu -- RMS norm of the query and key rows of each head, rotation by position, and
// quantize-append of the key and value rows, in one pass over a step's projections.
//
// For one row x of D elements (query or key of one head; w its norm's weights):
//   r = 1 / sqrt(sum(x^2) * (1/D) + eps),  y = (x * r) * w
//   pairs (y_a, y_b) of the first R elements:  (y_a c - y_b s,  y_b c + y_a s)
// with (c, s) from the row of the table at the token's position; the rest of y passes through.
// Pairs are (i, i + R/2), or (2i, 2i+1) when interleaved. A token may have a position on each of several
// axes (time, height, width): pair i then goes by the position on its axis. The result is rounded once to the
// input type; a key row then goes through the append's block rule (append.cu), as the rounded
// row would if it were handed to the append. Value rows are quantized as they are.
//
// All of it is binary32 with one rounding per operation and a fixed order of the sum of
// squares, so that the codes (which jump at the format's borders) are reproducible: eight
// squares t[i] += t[i+4], t[i+2], t[i+1]; the two groups of eight that rotate together are
// added; the D/16 pair sums, filled up with zeros to a power of two, add by halves.
//
// AXES: positions of several axes. A lane's pairs are four and four neighbours; where four are of one axis
// (sections of a multiple of four) they are one load as before.
//
// T = D/16 rounded up to a power of two lanes work on one row; lane j holds the two groups of
// eight elements that rotate together: groups j and j + R/16 below R/16, else 2j and 2j+1. A
// rotation then needs no exchange, and the sum of squares is in-lane plus log2(T) shuffles. A
// key row's 16-element blocks are put together through shared memory.
//
// A warp takes a token's rows a step at a time, 32/T rows to a step: first the query rows, then the
// key rows and the value rows (a step may hold some of both). What the rows share (the table's row, the weights,
// the page) is read once. With many tokens a warp has all steps of a token; with few, the steps
// are dealt out so that every step has a warp. Query rows are loaded two steps at a time.
//
// The floor is memory: the rows in, the queries and 9/16 byte a K/V element out. 32,764 tokens of 32
// query and 8 KV heads of 128 take 160 us (bf16, full rotation, 4.4 TB/s) and 178 us (fp16, 4over6,
// 4.0 TB/s); moving the data alone takes 119 us, and the instructions (some 150 of a warp for a step
// of two query rows) use 63 % of the issue slots beside it. Packed arithmetic (200 us), a cp.async
// ring (191), CTAs of 256 threads (207) and more CTAs an SM (179) do not overlap the two better. 64
// tokens take 4.7 us in a graph.
#include "internal.h"
#include "quantize.cuh"

namespace nvfp4 {
namespace {

constexpr int kThreads = 128;

// Exact binary32 values of eight packed elements.
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float x[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = BF16 ? __uint_as_float(w[k] << 16) : f32_from_f16_lo(w[k]);
    x[2 * k + 1] = BF16 ? f32_from_bf16_hi(w[k]) : f32_from_f16_hi(w[k]);
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float x[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] = BF16 ? bf16x2_from_f32(x[2 * k], x[2 * k + 1]) : f16x2_from_f32(x[2 * k], x[2 * k + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float sum_squares8(const float x[8]) {
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = __fmul_rn(x[i], x[i]);
#pragma unroll
  for (int h = 4; h >= 1; h /= 2) {
#pragma unroll
    for (int i = 0; i < h; ++i) t[i] = __fadd_rn(t[i], t[i + h]);
  }
  return t[0];
}

// (a c - b s, b c + a s), one rounding per operation.
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float ra = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = ra;
}

__device__ __forceinline__ void load4(const float* p, float v[4]) {
  const float4 f = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
}

// What a token's query and key rows share, in one lane: its groups, its part of the table's row.
struct Turn {
  int ga, gb;      // the lane's groups of eight
  bool turns;      // they are rotated
  float c[8], s[8];
};

template <bool BF16>
__device__ __forceinline__ void norm_rope(const NormRopeArgs& a, const Turn& turn, uint4 wa, uint4 wb,
                                          bool norm, int T, uint4& va, uint4& vb) {
  float xa[8], xb[8];
  unpack8<BF16>(va, xa);
  unpack8<BF16>(vb, xb);
  if (norm) {
    float sum = __fadd_rn(sum_squares8(xa), sum_squares8(xb));
    for (int o = T >> 1; o > 0; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xFFFFFFFFu, sum, o));
    const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, a.inv_d), a.eps)));
    float fa[8], fb[8];
    unpack8<BF16>(wa, fa);
    unpack8<BF16>(wb, fb);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      xa[e] = __fmul_rn(__fmul_rn(xa[e], r), fa[e]);
      xb[e] = __fmul_rn(__fmul_rn(xb[e], r), fb[e]);
    }
  }
  if (turn.turns) {
    if (a.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        rotate(xa[2 * e], xa[2 * e + 1], turn.c[e], turn.s[e]);
        rotate(xb[2 * e], xb[2 * e + 1], turn.c[4 + e], turn.s[4 + e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) rotate(xa[e], xb[e], turn.c[e], turn.s[e]);
    }
  }
  va = pack8<BF16>(xa);
  vb = pack8<BF16>(xb);
}

// MIXED: H is not a multiple of the rows of a step, and the value rows fill up the last key step: 62
// us against 74 with key and value rows in steps of their own (32,764 tokens, eight query heads and one KV head
// of 128, fp16, 4over6), 142 against 155 (24 and six). Where steps are full, choosing by lane would cost: 184 against 162
// (eight heads, bf16). Five CTAs to an SM serve the standard recipe's mixed steps (62 against 68 us);
// the same cap costs the others (66 against 62). AXES: five CTAs too, 171 us against 181 (32,764 tokens, bf16, three
// axes in sections of 16, 24 and 24 pairs) and 196 against 203 (fp16, 4over6, the axes of 32 pairs in turn, where a pair's
// cosine and sine are loads of their own).
// Where a lane's pairs begin is the same for all tokens, and is found before the loop over them; for bf16 and the recipes
// with binary16 errors inside it, where ptxas gives these instances 96 registers (five CTAs) in place of 111 (four): 173
// us against 193 (32,764 tokens, 32 query heads and eight KV heads of 128), with heads of 64 96 against 107, of 256 176
// against 198. The other recipes are faster the other way (bf16, binary32 errors: 178 against 198). A launch bound of five
// CTAs for all of them costs those that need none (169 against 162, standard recipe).
template <bool BF16, int MODE, bool MIXED, bool AXES>
__global__ void __launch_bounds__(kThreads, AXES || (MIXED && MODE == 0) ? 5 : 0) norm_rope_append_kernel(const NormRopeArgs a) {
  __shared__ Tables tab;
  __shared__ __align__(16) uint4 s_rows[kThreads / 32][64];  // a warp's rows, as groups of eight
  float gs[2];
  if (!load_scales(a.ap, gs)) return;
  fill_tables<MODE>(tab, gs);

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int T = 1 << a.log2_T, j = lane & (T - 1), nt = a.ap.D / 16, nr = a.rotary_dim / 16;
  const int per_step = 32 >> a.log2_T, slot_in_step = lane >> a.log2_T;
  const int32_t H = a.ap.H;
  const int64_t row = static_cast<int64_t>(a.ap.D) * 2;
  Turn turn;
  turn.turns = j < nr;
  turn.ga = j < nt ? (j < nr ? j : 2 * j) : 0;
  turn.gb = j < nt ? (j < nr ? j + nr : 2 * j + 1) : 0;
  constexpr bool kInLoop = !AXES && BF16 && MODE >= 3;
  int ca = 0, cb = 0;  // its pairs: four from each
  auto find_pairs = [&] {
    ca = a.interleaved ? 4 * turn.ga : 8 * j;
    cb = a.interleaved ? 4 * turn.gb : 8 * j + 4;
  };
  if (!kInLoop) find_pairs();
  uint32_t axes_a = 0, axes_b = 0;
  bool bad_axes = false;
  if (AXES && turn.turns) {
    axes_a = __ldg(reinterpret_cast<const uint32_t*>(a.pair_axes + ca));
    axes_b = __ldg(reinterpret_cast<const uint32_t*>(a.pair_axes + cb));
#pragma unroll
    for (int e = 0; e < 32; e += 8)
      bad_axes = bad_axes || (axes_a >> e & 0xFFu) >= a.axes || (axes_b >> e & 0xFFu) >= a.axes;
  }
  const int32_t k_end = a.q_steps + (H + per_step - 1) / per_step;  // steps from here on have value rows only
  const int64_t items = a.ap.nnz * a.parts;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + warp; item < items;
       item += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
    const int64_t i = div_q(item, a.div_parts);
    const int32_t from = static_cast<int32_t>(item - i * a.parts) * a.steps_per_part;
    const int32_t to = min(from + a.steps_per_part, a.q_steps + a.kv_steps);
    if (AXES) {
      // a row of the table for each axis: four pairs of one axis are a 16-byte load, mixed ones four loads
      bool in = !bad_axes;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t of = k ? axes_b : axes_a;
        const bool same = of == (of & 0xFFu) * 0x01010101u;
        int32_t p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = 0;
          if (turn.turns && !bad_axes && (e == 0 || !same))
            p[e] = __ldg(a.axis_positions + static_cast<int64_t>(of >> (8 * e) & 0xFFu) * a.ap.nnz + i);
          if (p[e] < 0 || p[e] >= a.num_positions) {
            in = false;
            p[e] = 0;
          }
        }
        if (!turn.turns || from >= k_end || !in) continue;
        const float* cs = a.cos_sin + (k ? cb : ca);
        if (same) {
          cs += static_cast<int64_t>(p[0]) * a.rotary_dim;
          load4(cs, turn.c + 4 * k);
          load4(cs + a.rotary_dim / 2, turn.s + 4 * k);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float* at = cs + static_cast<int64_t>(p[e]) * a.rotary_dim + e;
            turn.c[4 * k + e] = __ldg(at);
            turn.s[4 * k + e] = __ldg(at + a.rotary_dim / 2);
          }
        }
      }
      if (__any_sync(0xFFFFFFFFu, !in)) {
        if (lane == 0) flag(a.ap.status, NVFP4_DEV_BAD_POSITION);
        continue;
      }
    } else {
      const int32_t pos = __ldg(a.ap.positions + i);
      if (nr > 0 && (pos < 0 || pos >= a.num_positions)) {
        if (lane == 0) flag(a.ap.status, NVFP4_DEV_BAD_POSITION);
        continue;
      }
      if (turn.turns && from < k_end) {
        const float* cs = a.cos_sin + static_cast<int64_t>(pos) * a.rotary_dim;
        const float* sn = cs + a.rotary_dim / 2;
        if (kInLoop) find_pairs();
        load4(cs + ca, turn.c);
        load4(cs + cb, turn.c + 4);
        load4(sn + ca, turn.s);
        load4(sn + cb, turn.s + 4);
      }
    }
    if (from < a.q_steps) {
      uint4 wa{}, wb{};
      if (a.q_weight) {
        wa = __ldg(reinterpret_cast<const uint4*>(a.q_weight) + turn.ga);
        wb = __ldg(reinterpret_cast<const uint4*>(a.q_weight) + turn.gb);
      }
      const uint8_t* src = a.q + i * a.q_row_bytes;
      uint8_t* dst = a.q_out + i * a.q_out_row_bytes;
      const int32_t end = min(to, a.q_steps);
      for (int32_t step = from; step < end; step += 2) {
        uint4 v[2][2] = {};
        bool live[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int32_t h = (step + k) * per_step + slot_in_step;
          live[k] = step + k < end && h < a.Hq && j < nt;
          if (live[k]) {
            const uint4* x = reinterpret_cast<const uint4*>(src + h * row);
            v[k][0] = x[turn.ga];
            v[k][1] = x[turn.gb];
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (step + k >= end) break;
          norm_rope<BF16>(a, turn, wa, wb, a.q_weight != nullptr, T, v[k][0], v[k][1]);
          if (live[k]) {
            uint4* y = reinterpret_cast<uint4*>(dst + ((step + k) * per_step + slot_in_step) * row);
            y[turn.ga] = v[k][0];
            y[turn.gb] = v[k][1];
          }
        }
      }
    }
    if (to <= a.q_steps) continue;
    const RowMeta m = resolve_row(a.ap, i);
    uint4 wa{}, wb{};
    if (a.k_weight && from < k_end) {
      wa = __ldg(reinterpret_cast<const uint4*>(a.k_weight) + turn.ga);
      wb = __ldg(reinterpret_cast<const uint4*>(a.k_weight) + turn.gb);
    }
#pragma unroll 1
    for (int32_t step = max(from, a.q_steps); step < to; ++step) {
      const int32_t w0 = (step - a.q_steps) * per_step, w = w0 + slot_in_step;  // the K rows, then the V rows
      const int kv = (MIXED ? w : w0) >= H;
      const int32_t h = w - kv * H;
      const bool live = (!MIXED || w < 2 * H) && j < nt;
      const uint8_t* src = (kv ? a.ap.v + i * a.ap.v_row_bytes : a.ap.k + i * a.ap.k_row_bytes) + h * row;
      uint4 lo{}, hi{};
      auto load = [&](int ga, int gb) {
        if (live) {
          lo = reinterpret_cast<const uint4*>(src)[ga];
          hi = reinterpret_cast<const uint4*>(src)[gb];
        }
      };
      auto norm_key = [&](uint4& ya, uint4& yb) {
        norm_rope<BF16>(a, turn, wa, wb, a.k_weight != nullptr, T, ya, yb);
        if (nr > 0) {  // groups back into blocks
          uint4* buf = s_rows[warp] + (lane - j) * 2;
          __syncwarp();
          if (j < nt) {
            buf[turn.ga] = ya;
            buf[turn.gb] = yb;
          }
          __syncwarp();
          ya = buf[2 * j];
          yb = buf[2 * j + 1];
        }
      };
      if constexpr (MIXED) {
        load(kv ? 2 * j : turn.ga, kv ? 2 * j + 1 : turn.gb);
        if (step < k_end) {
          uint4 ya = lo, yb = hi;
          norm_key(ya, yb);
          if (!kv) {
            lo = ya;
            hi = yb;
          }
        }
      } else if (kv) {
        load(2 * j, 2 * j + 1);
      } else {
        load(turn.ga, turn.gb);
        norm_key(lo, hi);
      }
      if (live && (m.flags & (1 << kv))) {
        U32x8 in;
        in.w[0] = lo.x; in.w[1] = lo.y; in.w[2] = lo.z; in.w[3] = lo.w;
        in.w[4] = hi.x; in.w[5] = hi.y; in.w[6] = hi.z; in.w[7] = hi.w;
        const BlockOut q = quantize_block<BF16, MODE>(in, make_consts(kv ? gs[1] : gs[0]), tab, kv, a.ap.cap_a,
                                                      a.ap.neg_zero);
        const nvfp4_paged_cache& c = kv ? a.ap.vc : a.ap.kc;
        const int64_t r = a.ap.layout == NVFP4_NHD ? static_cast<int64_t>(m.slot) * H + h
                                                   : static_cast<int64_t>(h) * a.ap.ps + m.slot;
        uint8_t* dst = c.data + m.page * c.data_page_stride + r * (a.ap.D / 2) + 8 * j;
        *reinterpret_cast<uint2*>(dst) = make_uint2(q.c0, q.c1);
        c.sf[m.page * c.sf_page_stride + r * nt + j] = static_cast<uint8_t>(q.s);
      }
    }
  }
}

template <bool BF16, int MODE, bool AXES>
nvfp4_status launch_t(NormRopeArgs a, cudaStream_t stream) {
  const int per_step = 32 >> a.log2_T;
  const auto kern = a.ap.H % per_step != 0 ? norm_rope_append_kernel<BF16, MODE, true, AXES>
                                           : norm_rope_append_kernel<BF16, MODE, false, AXES>;
  int64_t cap;
  if (nvfp4_status st = resident_ctas(reinterpret_cast<const void*>(kern), kThreads, 0, 32,
                                      "nvfp4_qk_norm_rope_append_paged", &cap))
    return st;
  a.q_steps = (a.Hq + per_step - 1) / per_step;
  a.kv_steps = (2 * a.ap.H + per_step - 1) / per_step;
  // parts of a token: enough that the warps of one wave have an item each
  const int64_t warps = cap * (kThreads / 32);
  const int32_t steps = a.q_steps + a.kv_steps;
  const int64_t wanted = (warps + a.ap.nnz - 1) / a.ap.nnz;
  a.parts = static_cast<int32_t>(wanted < steps ? wanted : steps);
  a.steps_per_part = (steps + a.parts - 1) / a.parts;
  a.parts = (steps + a.steps_per_part - 1) / a.steps_per_part;
  a.div_parts = make_div(a.parts);
  const int64_t need = (a.ap.nnz * a.parts + kThreads / 32 - 1) / (kThreads / 32);
  const int grid = static_cast<int>(need < cap ? need : cap);
  kern<<<grid, kThreads, 0, stream>>>(a);
  return check_launch("nvfp4_qk_norm_rope_append_paged");
}

template <bool BF16, bool AXES>
nvfp4_status launch_m(const NormRopeArgs& a, int mode, cudaStream_t s) {
  switch (mode) {
    case 0: return launch_t<BF16, 0, AXES>(a, s);
    case 1: return launch_t<BF16, 1, AXES>(a, s);
    case 2: return launch_t<BF16, 2, AXES>(a, s);
    case 3: return launch_t<BF16, 3, AXES>(a, s);
    default: return launch_t<BF16, 4, AXES>(a, s);
  }
}

}  // namespace

nvfp4_status launch_norm_rope_append(const NormRopeArgs& a, bool bf16, int mode,
                                     cudaStream_t stream) {
  if (a.axis_positions)
    return bf16 ? launch_m<true, true>(a, mode, stream) : launch_m<false, true>(a, mode, stream);
  return bf16 ? launch_m<true, false>(a, mode, stream) : launch_m<false, false>(a, mode, stream);
}

}  // namespace nvfp4
