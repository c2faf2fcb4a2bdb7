// Attention with a learned relative position bias by buckets: what its
// kernels share (matrix fragments, tiles in LDS, the bias window).
//
//   s_ij = scale q_i.k_j + table[map[clamp(j - pos_i, -far, far)]][head]
//   p_ij = exp(s_ij - lse_i) over the keys that query i sees,  o_i = sum p_ij v_j
//   dv_j = sum p_ij do_i,  dp_ij = do_i.v_j,  ds_ij = p_ij (dp_ij - delta_i),
//   delta_i = do_i.o_i,  dq_i = scale sum ds_ij k_j,  dk_j = scale sum ds_ij q_i,
//   dtable[b][head] = sum of ds_ij over the pairs of bucket b
//
// Matrix products run on 32x32x16 MFMAs.  Lane l = 32 h + n of a fragment holds
// row (or column) n and the 8 contraction indices of half h.  A result's lane
// holds column n and rows 8 (r / 4) + 4 h + r % 4 for its 16 registers r.
//
// float32 values are taken apart into three bfloat16 ones, x = a + b + c exactly
// (8 significant bits each, rounded to nearest, so that the rests have either
// sign), and a product is the six terms a a', a b', b a', a c', c a', b b' with
// float32 sums; what is left out, b c' + c b' + c c', is at most 2^-24 of x x'.
// Six bfloat16 products of 8 passes take the place of eight float32 ones of 16.
//
// Probabilities never pass through LDS: their product with the next operand
// contracts over the result's rows, in whatever order, as long as the other
// operand is read in that order too.  Registers 8 c .. 8 c + 7 of a lane are
// its 8 contraction indices of step c: rows 16 c + 4 h + 0..3 and 16 c + 8 + 4 h
// + 0..3.  The other operand comes out of a row-major LDS tile column by
// column in exactly these rows, with the transposing LDS read for 16-bit types.
#pragma once

#include "fm_op.h"

namespace fm {

typedef float acc16 __attribute__((ext_vector_type(16)));
typedef float acc4 __attribute__((ext_vector_type(4)));
typedef short short4v __attribute__((ext_vector_type(4)));

template <class T>
struct RawOf {
  typedef T type __attribute__((ext_vector_type(8)));
};
template <class T>
using Raw = typename RawOf<T>::type;  // eight values as they are in memory
struct Frag3 {
  Raw<bf16_t> a, b, c;
};
template <class T>
struct FragOf {
  typedef Raw<T> type;
  typedef T lds;  // element of an LDS tile
  static constexpr int planes = 1;
};
template <>
struct FragOf<float> {
  typedef Frag3 type;
  typedef bf16_t lds;
  static constexpr int planes = 3;
};
template <class T>
using Frag = typename FragOf<T>::type;
template <class T>
using Lds = typename FragOf<T>::lds;

// N float32 values as three times N bfloat16 ones.  An infinity stays one.
template <int N, bool INF>
__device__ __forceinline__ void take_apart(const float (&x)[N], bf16_t (&a)[N], bf16_t (&b)[N],
                                           bf16_t (&c)[N]) {
  typedef float fN __attribute__((ext_vector_type(N)));
  typedef bf16_t bN __attribute__((ext_vector_type(N)));
  fN v, r;
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = x[e];
  const bN va = __builtin_convertvector(v, bN);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float w = (float)va[e];
    r[e] = INF && __builtin_isinf(w) ? 0.f : v[e] - w;
  }
  const bN vb = __builtin_convertvector(r, bN);
#pragma unroll
  for (int e = 0; e < N; ++e) r[e] -= (float)vb[e];
  const bN vc = __builtin_convertvector(r, bN);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    a[e] = va[e];
    b[e] = vb[e];
    c[e] = vc[e];
  }
}
template <bool INF>
__device__ __forceinline__ Frag3 take_apart(const Raw<float>& x) {
  float v[8];
  bf16_t a[8], b[8], c[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = x[e];
  take_apart<8, INF>(v, a, b, c);
  Frag3 f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    f.a[e] = a[e];
    f.b[e] = b[e];
    f.c[e] = c[e];
  }
  return f;
}
__device__ __forceinline__ Raw<bf16_t> to_frag(Raw<bf16_t> x) { return x; }
__device__ __forceinline__ Raw<f16_t> to_frag(Raw<f16_t> x) { return x; }
__device__ __forceinline__ Frag3 to_frag(Raw<float> x) { return take_apart<true>(x); }

__device__ __forceinline__ acc16 mma32(Raw<bf16_t> a, Raw<bf16_t> b, acc16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ acc16 mma32(Raw<f16_t> a, Raw<f16_t> b, acc16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ acc16 mma32(const Frag3& x, const Frag3& y, acc16 c) {
  c = mma32(x.b, y.b, c);
  c = mma32(x.c, y.a, c);
  c = mma32(x.a, y.c, c);
  c = mma32(x.b, y.a, c);
  c = mma32(x.a, y.b, c);
  return mma32(x.a, y.a, c);
}
// 16x16x32: lane 16 g + n holds row n and the 8 contraction indices of quarter
// g; a result's lane column n, rows 4 g + r.
__device__ __forceinline__ acc4 mma16(Raw<bf16_t> a, Raw<bf16_t> b, acc4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ acc4 mma16(Raw<f16_t> a, Raw<f16_t> b, acc4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ acc4 mma16(const Frag3& x, const Frag3& y, acc4 c) {
  c = mma16(x.b, y.b, c);
  c = mma16(x.c, y.a, c);
  c = mma16(x.a, y.c, c);
  c = mma16(x.b, y.a, c);
  c = mma16(x.a, y.b, c);
  return mma16(x.a, y.a, c);
}

// Eight contiguous elements of a row in memory, of which `have` exist.
template <class T>
__device__ __forceinline__ Raw<T> load_raw(const T* p, int have) {
  Raw<T> f;
  if (have >= 8) {
    __builtin_memcpy(&f, p, sizeof(f));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = e < have ? p[e] : (T)0.f;
  }
  return f;
}

// Rows of a matrix [.., dim] in memory, for fragments of eight elements: VEC
// (whole, aligned 16-byte groups, see attn_groups) without a branch, by buffer
// loads whose offsets lie past the range where nothing is.  A branch per
// fragment makes the kernels' prologues long: mostly skipped code, but fetched.
template <class T, bool VEC>
struct Rows {
  const T* base;
  int64_t stride;
  int count, dim;  // rows that exist
  __device__ __forceinline__ Raw<T> at(int row, int d) const {
    if constexpr (VEC) {
      typedef uint32_t u4 __attribute__((ext_vector_type(4)));
      const __amdgpu_buffer_rsrc_t r =
          __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, 0x7ffffff0, 0x00020000);
      struct Parts {
        u4 v[sizeof(Raw<T>) / 16];
      } p;
#pragma unroll
      for (int k = 0; k < (int)(sizeof(Raw<T>) / 16); ++k) {
        const int e = d + k * Vec16<T>::n;
        const uint32_t off = (uint32_t)((row * stride + e) * sizeof(T));
        p.v[k] = __builtin_amdgcn_raw_buffer_load_b128(
            r, row >= 0 && row < count && e < dim ? off : 0x7ffffff0u, 0, 0);
      }
      return __builtin_bit_cast(Raw<T>, p);
    } else {
      return load_raw(base + row * stride + d, row >= 0 && row < count ? dim - d : 0);
    }
  }
};

// Row-major LDS tile: 16 bytes of padding per row spread the rows over the
// banks.  float32: three planes of 32 rows.
template <class T, int DP>
struct Tile {
  static constexpr int ld = DP + 8;
  static constexpr int plane = 32 * ld;
  static constexpr int chunks = DP * (int)sizeof(T) / 16;  // 16-byte groups of a row in memory
  static constexpr int size(int rows) { return FragOf<T>::planes * rows * ld; }
};

// Fragment of row n (a lane's own), contraction indices 16 s + 8 h ..: one
// 16-byte read.
template <class T, int DP>
__device__ __forceinline__ Frag<T> tile_rows(const Lds<T>* tile, int row, int s, int h) {
  const Lds<T>* p = tile + row * Tile<T, DP>::ld + 16 * s + 8 * h;
  if constexpr (sizeof(T) == 4)
    return {*(const Raw<bf16_t>*)p, *(const Raw<bf16_t>*)(p + Tile<T, DP>::plane),
            *(const Raw<bf16_t>*)(p + 2 * Tile<T, DP>::plane)};
  else
    return *(const Frag<T>*)p;
}

// Four rows of a column each, twice: `p` and `step` elements further.
__device__ __forceinline__ short4v lds_read_tr(const void* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4v*)p);
}
template <class E>
__device__ __forceinline__ Raw<E> lds_columns(const E* p, int step) {
  typedef short short8v __attribute__((ext_vector_type(8)));
  const short4v lo = lds_read_tr(p), hi = lds_read_tr(p + step);
  const short8v both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(Raw<E>, both);
}
template <class T>
__device__ __forceinline__ Frag<T> lds_columns_of(const Lds<T>* p, int step, int plane) {
  if constexpr (sizeof(T) == 4)
    return {lds_columns(p, step), lds_columns(p + plane, step), lds_columns(p + 2 * plane, step)};
  else
    return lds_columns(p, step);
}
// Fragment of column d0 + l % 32, contraction over rows r0 + 4 h + 0..3 and
// r0 + 8 + 4 h + 0..3: a group of 16 lanes reads 4 rows of 16 columns, 8 bytes
// each, and gets them transposed, lane i the 4 rows of column i.
template <class T, int DP>
__device__ __forceinline__ Frag<T> tile_cols(const Lds<T>* tile, int r0, int d0, int lane) {
  constexpr int ld = Tile<T, DP>::ld;
  const int g = lane >> 4, i = lane & 15;
  return lds_columns_of<T>(tile + (r0 + 4 * (g >> 1) + (i >> 2)) * ld + d0 + 16 * (g & 1) + 4 * (i & 3),
                           8 * ld, Tile<T, DP>::plane);
}

// Eight float32 values as a fragment.
template <class T>
__device__ __forceinline__ Frag<T> round_frag(const Raw<float>& v) {
  if constexpr (sizeof(T) == 4)
    return take_apart<false>(v);
  else
    return __builtin_convertvector(v, Raw<T>);
}
// Registers 8 c .. 8 c + 7 of a result as the fragment of contraction step c.
template <class T>
__device__ __forceinline__ Frag<T> acc_frag(const acc16& a, int c) {
  Raw<float> v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = a[8 * c + e];
  return round_frag<T>(v);
}

// 16 bytes of a row in memory into its place in a tile.
template <class T, int DP>
__device__ __forceinline__ void tile_put(Lds<T>* tile, int row, int col, const Vec16<T>& v) {
  Lds<T>* p = tile + row * Tile<T, DP>::ld + col;
  if constexpr (sizeof(T) == 4) {
    struct Four {
      bf16_t v[4];
    };
    Four a, b, c;
    take_apart<4, true>(v.v, a.v, b.v, c.v);
    *(Four*)__builtin_assume_aligned(p, 8) = a;
    *(Four*)__builtin_assume_aligned(p + Tile<T, DP>::plane, 8) = b;
    *(Four*)__builtin_assume_aligned(p + 2 * Tile<T, DP>::plane, 8) = c;
  } else {
    *(Vec16<T>*)__builtin_assume_aligned(p, 16) = v;
  }
}

// A tile of ROWS rows on its way from memory to LDS.  Rows from `valid` on and
// columns from `dim` on become zero; nothing past them is read.
//
// VEC (rows of whole, aligned 16-byte groups): buffer loads whose range ends
// with the last valid row, so that neither end costs an instruction, held in
// registers until store().  A thread's groups lie a whole number of rows apart
// where they can: then one offset serves all, with the step as the load's
// scalar offset.
template <class T, int DP, int ROWS, int NT, bool VEC>
struct TileLoad {
  static constexpr int ch = Tile<T, DP>::chunks;
  static constexpr int n = (ROWS * ch + NT - 1) / NT;
  static constexpr int ve = Vec16<T>::n;
  static constexpr bool even = NT % ch == 0 && ROWS % (NT / ch) == 0;
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  u4 v[n];
  uint32_t at[even ? 1 : n];
  uint32_t step;
  __device__ __forceinline__ void init(int64_t stride, int dim, int tid) {
    step = even ? (uint32_t)(NT / ch * stride * sizeof(T)) : 0u;
#pragma unroll
    for (int i = 0; i < (even ? 1 : n); ++i) {
      const int c = i * NT + tid, row = c / ch, col = (c - row * ch) * ve;
      at[i] = row < ROWS && col < dim ? (uint32_t)((row * stride + col) * sizeof(T)) : 0x7ffffff0u;
    }
  }
  __device__ __forceinline__ void load(const T* base, int64_t stride, int valid, int dim, int tid) {
    const int rows = valid < ROWS ? valid : ROWS;
    const int bytes = rows <= 0 ? 0 : (int)(((rows - 1) * stride + dim) * sizeof(T));
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, bytes, 0x00020000);
#pragma unroll
    for (int i = 0; i < n; ++i)
      v[i] = __builtin_amdgcn_raw_buffer_load_b128(r, at[even ? 0 : i], even ? i * step : 0, 0);
  }
  __device__ __forceinline__ void store(Lds<T>* tile, int tid) const {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int c = i * NT + tid, row = c / ch, col = (c - row * ch) * ve;
      if (ROWS * ch % NT == 0 || row < ROWS)
        tile_put<T, DP>(tile, row, col, __builtin_bit_cast(Vec16<T>, v[i]));
    }
  }
};
// Rows of any width, stride and alignment: nothing is held, store() copies
// group by group.
template <class T, int DP, int ROWS, int NT>
struct TileLoad<T, DP, ROWS, NT, false> {
  static constexpr int ch = Tile<T, DP>::chunks;
  static constexpr int ve = Vec16<T>::n;
  const T* base;
  int64_t stride;
  int valid, dim;
  __device__ __forceinline__ void init(int64_t, int, int) {}
  __device__ __forceinline__ void load(const T* base_, int64_t stride_, int valid_, int dim_, int) {
    base = base_;
    stride = stride_;
    valid = valid_;
    dim = dim_;
  }
  __device__ __forceinline__ void store(Lds<T>* tile, int tid) const {
#pragma unroll 1
    for (int c = tid; c < ROWS * ch; c += NT) {
      const int row = c / ch, col = (c - row * ch) * ve;
      tile_put<T, DP>(tile, row, col,
                      load16_part(base + row * stride + col, row < valid ? dim - col : 0, (T)0.f));
    }
  }
};

// Waves per SIMD the big kernels are compiled for.  Two keep their registers
// within 256, which the products' results then share with the vector unit;
// beyond, the compiler moves every score between the two register files.
// float32 fragments of more than 64 columns do not fit.
template <class T, int DP>
constexpr int attn_waves() { return sizeof(T) == 2 || DP == 64 ? 2 : 1; }

// Bias by distance, as the accumulators' start: table value / scale, so that
// one multiplication scales both.  The window covers every distance of a
// 32x32 tile that reaches inside +-far (kBiasPad more on either side); tiles
// beyond take an end value.
// Finite table values count as at most 2^16 either way (float16's whole range):
// enough to hide a key beside any other, while the scores of a row whose keys all
// have such a value, and its log sum exp, still hold the products' part in float32
// (half a step there is 2^-8).  Larger ones, the masks of a type's lowest value,
// would leave nothing of it, or float32's range by the factor 1 / scale or log2 e.
constexpr float kBiasMost = 65536.f;
template <class T>
__device__ __forceinline__ float bias_of_bucket(const AttnArgs& a, int head, int b) {
  if (b < 0 || b >= a.num_buckets) return 0.f;  // a distance without a bucket
  const int64_t at = (int64_t)b * a.heads + head;
  const float v = a.table32 ? ((const float*)a.table)[at] : (float)((const T*)a.table)[at];
  return __builtin_isfinite(v) ? fminf(fmaxf(v, -kBiasMost), kBiasMost) : v;
}
template <class T>
__device__ __forceinline__ float bias_of(const AttnArgs& a, int head, int d) {
  const int i = d < -a.far ? 0 : d > a.far ? 2 * a.far : d + a.far;
  return bias_of_bucket<T>(a, head, a.map[i]);
}

__device__ __forceinline__ int clamp_int(int v, int lo, int hi) {
  return v < lo ? lo : v > hi ? hi : v;
}
__device__ __forceinline__ int key_count(const AttnArgs& a, int b) {
  return a.key_lengths ? clamp_int(a.key_lengths[b], 0, a.k_len) : a.k_len;
}
__device__ __forceinline__ int position_of_first(const AttnArgs& a, int b) {
  const int o = a.query_offset ? a.query_offset[b] : a.query_offset_value;
  return clamp_int(o, -(1 << 30), 1 << 30);
}

// The distances up to `left` share the first bucket of the map and those from
// `right` on its last (the ends may be wide buckets: 32 of them up to distance
// 128 leave 91 to 128 to the last).  A 32x32 tile, dist = first key - first
// query's position, that lies in one of them has one bias for every pair; in the
// others the window's values start the accumulators.
struct Reach {
  int left, right;
};
__device__ __forceinline__ bool tile_before(int dist, Reach r) { return dist + 31 <= r.left; }
__device__ __forceinline__ bool tile_behind(int dist, Reach r) { return dist - 31 >= r.right; }
// Rows keys, columns queries: rows 8 (r / 4) + 4 h + r % 4, column n have
// distance dist + row - n.
__device__ __forceinline__ acc16 bias_start_keys(const float* bias, int far, int dist, int h, int n) {
  const float* p = bias + dist + far + kBiasPad + 4 * h - n;
  acc16 acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = p[8 * (r / 4) + r % 4];
  return acc;
}
// Rows queries, columns keys: distance dist + n - row.
__device__ __forceinline__ acc16 bias_start_queries(const float* bias, int far, int dist, int h, int n) {
  const float* p = bias + dist + far + kBiasPad - 4 * h + n;
  acc16 acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = p[-(8 * (r / 4) + r % 4)];
  return acc;
}
// An accumulator whose rows start at the values of an LDS row vector.
__device__ __forceinline__ acc16 acc_rows(const float* p, int h) {
  acc16 a;
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const float4 v = *(const float4*)(p + 8 * y + 4 * h);
    a[4 * y] = v.x;
    a[4 * y + 1] = v.y;
    a[4 * y + 2] = v.z;
    a[4 * y + 3] = v.w;
  }
  return a;
}
__device__ __forceinline__ acc16 acc_zero() {
  acc16 a;
#pragma unroll
  for (int r = 0; r < 16; ++r) a[r] = 0.f;
  return a;
}

// Fills the window; a thread's map entries are on their way together, and then
// its table entries.  `ends` gets each wave's part of the map's reach (2 values).
template <class T, bool REACH = true>
__device__ __forceinline__ void fill_bias(const AttnArgs& a, int head, float* bias, float* ends, int tid, int nt) {
  const float inv = 1.f / a.scale;
  const int win = bias_window(a.far), first = a.map[0], last = a.map[2 * a.far];
  float below = -0x1p29f, above = -0x1p29f;  // the farthest distances of other buckets, below negated
  for (int i0 = tid; i0 < win; i0 += 4 * nt) {
    int b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) b[k] = a.map[clamp_int(min(i0 + k * nt, win - 1) - kBiasPad, 0, 2 * a.far)];
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float d = (float)(min(i0 + k * nt, win - 1) - a.far - kBiasPad);
      v[k] = bias_of_bucket<T>(a, head, b[k]);
      if constexpr (REACH) {
        below = fmaxf(below, b[k] != first ? -d : below);
        above = fmaxf(above, b[k] != last ? d : above);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + k * nt < win) bias[i0 + k * nt] = v[k] * inv;
  }
  if constexpr (!REACH) return;
  below = lanes_max<64>(below);
  above = lanes_max<64>(above);
  if ((tid & 63) == 0) {
    ends[2 * (tid >> 6)] = below;
    ends[2 * (tid >> 6) + 1] = above;
  }
}
// From the four waves' parts, after a barrier.
__device__ __forceinline__ Reach reach_of(const float* ends) {
  const float below = fmaxf(fmaxf(ends[0], ends[2]), fmaxf(ends[4], ends[6]));
  const float above = fmaxf(fmaxf(ends[1], ends[3]), fmaxf(ends[5], ends[7]));
  return {__builtin_amdgcn_readfirstlane(-(int)below - 1), __builtin_amdgcn_readfirstlane((int)above + 1)};
}

// Which unit (entry, key head) and which of its blocks a workgroup takes.
// Workgroups go round the 8 XCDs one by one; where the units divide among them,
// an XCD keeps whole units, whose keys and values then stay in its L2.  Units
// go round the XCDs too: the heads of a long entry would otherwise share one
// XCD.  8 entries of 1501 to 845 keys, 16 heads, 64 columns, bf16, us: forward 86,
// whole entries per XCD 102, blocks in order 91; backward 292, in order 307; 1 x 8
// heads x 8000: 185 and 189; 9 x 8 x 1000: 37.5 and 40.9.
struct Place {
  int unit, block;
  bool none;
};
// Few units that do not divide among the XCDs would leave some of them idle.
__host__ __device__ inline bool place_by_xcd(int64_t units) { return units % 8 == 0 || units >= 64; }
__device__ __forceinline__ Place place_of(int units, int blocks, int id) {
  if (place_by_xcd(units)) {
    const int t = id >> 3, u = t / blocks * 8 + (id & 7);
    return {u, t % blocks, u >= units};
  }
  return {id / blocks, id % blocks, id / blocks >= units};
}
inline unsigned place_grid(int64_t units, int64_t blocks) {
  return (unsigned)(place_by_xcd(units) ? (units + 7) / 8 * 8 * blocks : units * blocks);
}

__device__ __forceinline__ int64_t attn_row_count(const AttnArgs& a) {
  return (int64_t)a.batch * a.heads * a.q_len;
}

// The wave of a thread as a scalar: what depends on it alone then branches
// without touching the lane mask.
__device__ __forceinline__ int wave_index() {
  return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
}

__device__ __forceinline__ float as_scalar(float x) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

// The same value to the compiler as a new one: what is computed from it after
// a loop is not kept in registers across the loop.
__device__ __forceinline__ int afresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Over the two halves of a wave, in every lane.
__device__ __forceinline__ float halves_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float halves_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// A border for the compiler's scheduler, which by itself puts every LDS read
// right before the product that waits for it.  The kernels read the operands of
// one stage's products in the stage before.
__device__ __forceinline__ void stage() { __builtin_amdgcn_sched_barrier(0); }
// Within a stage: N times a product and VALU vector instructions.
template <int N, int VALU>
__device__ __forceinline__ void alternate() {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
  }
}

// N steps that each use an operand from LDS.  float32's six terms last as long
// as a read takes: there each step's operand is read in the step before.
template <class T, int N, class Read, class Use>
__device__ __forceinline__ void steps(const Read& read, const Use& use) {
  if constexpr (sizeof(T) == 4) {
    Frag<T> f[2];
    f[0] = read(0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i + 1 < N) f[(i + 1) & 1] = read(i + 1);
      stage();
      use(i, f[i & 1]);
      stage();
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) use(i, read(i));
  }
}

// Stores 4 consecutive elements of a result column's rows (VEC: all of them
// exist).
template <class T, bool VEC>
__device__ __forceinline__ void store4(T* p, float a, float b, float c, float d, int have) {
  typedef T t4 __attribute__((ext_vector_type(4)));
  typedef float f4 __attribute__((ext_vector_type(4)));
  const f4 v = {a, b, c, d};
  const t4 r = __builtin_convertvector(v, t4);
  if (VEC || have >= 4) {
    __builtin_memcpy(p, &r, sizeof(r));
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < have) p[e] = r[e];
  }
}

}  // namespace fm
