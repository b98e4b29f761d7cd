// Norm and rotary position of heads in one pass, and the same on the way into
// the paged MXFP4 cache.
//
//   n = x / sqrt(mean(x^2) + eps) * w            over a head, where there is a w
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t)   for each pair of the head
//
// A pair's angle is position * frequency.  Positions reach far beyond what a
// binary32 product keeps of its fraction, so frequencies are whole numbers of
// 2^-64 turns: the product modulo 2^64 is the angle's fraction of a turn, exact
// but for the frequency's own rounding, and one 64-bit multiplication.
//
// A warp takes (a slice of) one token's heads.  Its lanes work out the token's
// cosines and sines once, 32 pairs at a time, and pass them through shared
// memory; then 32 / L heads go at a time, L = dim / 16 lanes a head.  A lane holds two chunks of eight elements: in halves
// pairs (i, i + rot / 2) chunk c and chunk c + rot / 16, so that both elements
// of a pair meet in one lane without a shuffle; neighbours are in one chunk
// anyway, and the chunks lie dim / 2 apart, so that the lanes of a load are
// side by side either way.  Sums are binary32; the result is rounded once, to
// the output's type or to MXFP4.
//
// What goes into the cache needs the largest of 32 elements, four chunks: those of
// four neighbouring lanes, or, where only part of a head is rotated, of any, whose
// maxima then go through shared memory.
//
// What bounds it: HBM, 37,810 tokens of 84 heads of 128 in BF16 (1.63 GB) in 264 us,
// 91% of the copy rate (FP32: 94%; without a norm 96%); with few heads or narrow ones a
// token's own work, its angles and their products with the weights, which takes a warp
// about as long as five steps of heads (60,000 tokens of 40 heads of 64: 125 us, 73%).
// Registers decide: with 96 two heads' loads are under way and next to nothing spills;
// ten blocks an SM 264 us, eight 287, nine 275, eleven 346.  Into the cache 37,810 tokens
// of 32 + 8 + 8 heads (0.82 GB) 159 us in neighbouring pairs and 167 in halves, where
// rotating queries and keys and then writing the cache take 132 + 37; twelve blocks an
// SM, ten 169 and 173, eight 196.  Several tokens to a warp, in turn: 271 to 293 us for
// the first.  One token: 2.9 us.
#include <string>
#include <type_traits>

#include "mx_common.cuh"

namespace nvfp4 {

nvfp4_status check_cache(const mxfp4_cache* cache, int* page_shift, const std::string& nm);

namespace {

constexpr int kThreads = 64;  // small blocks, as warps end when their token does (256 threads: 2% slower)
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 128;

struct Rows {  // heads of one kind
  const void* x;
  void* out;
  const void* weight;
  int64_t st, sh, o_st, o_sh;
  int64_t step, o_step;  // strides of a warp's step: the heads that it takes at a time
  int32_t heads;
  int32_t steps;  // heads / (heads at a time), rounded up
};

struct RotaryParams {
  Rows rows[3];  // queries, keys, values
  const int64_t* turns;
  const int32_t* axis;
  const int32_t* positions;
  int32_t pairs, axes, dim;
  int32_t lanes, at_once;  // of a head; heads of a warp
  int32_t wide_weights;  // the weights are binary32, the heads are not
  int32_t weight_vec;    // 16-byte accesses to them are aligned
  float eps, inv_dim;
  int64_t tokens;
  int32_t slices, per_slice;  // of a token's steps
  // of the cache
  const int64_t* slots;
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int64_t pages;
  int32_t page_shift, kv_heads;
};

// cos and sin of a fraction of a turn in 2^-64: the nearest quarter turn first,
// then at most an eighth, of which binary32 keeps 2^-28.
__device__ __forceinline__ float2 turn_to_cos_sin(uint64_t turn) {
  const uint32_t t = uint32_t((turn + 0x80000000ull) >> 32);
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  const int32_t rest = int32_t(t - (quarter << 30));
  float s, c;
  sincospif(float(rest) * 0x1p-31f, &s, &c);
  const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
  return make_float2((quarter + 1) & 2 ? -x : x, quarter & 2 ? -y : y);
}

// Eight elements as loaded.
template <typename T>
struct Chunk8 {
  uint32_t w[int(sizeof(T)) * 2];
};
template <typename T, bool kVec>
__device__ __forceinline__ Chunk8<T> load_chunk(const T* p) {
  Chunk8<T> r;
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r.w[i] = uint32_t(reinterpret_cast<const uint16_t*>(p)[2 * i]) |
               uint32_t(reinterpret_cast<const uint16_t*>(p)[2 * i + 1]) << 16;
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void unpack(const Chunk8<T>& r, float* f) {
#pragma unroll
  for (int i = 0; i < int(sizeof(T)) * 2; ++i) {
    if constexpr (sizeof(T) == 4) {
      f[i] = __uint_as_float(r.w[i]);
    } else {
      const float2 t = word_to_f32<T>(r.w[i]);
      f[2 * i] = t.x, f[2 * i + 1] = t.y;
    }
  }
}
template <typename T, bool kVec>
__device__ __forceinline__ void store_chunk(T* p, const float* f) {
  if constexpr (!kVec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = from_f32<T>(f[i]);
  } else if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(f32_to_word<T>(f[0], f[1]), f32_to_word<T>(f[2], f[3]),
                                              f32_to_word<T>(f[4], f[5]), f32_to_word<T>(f[6], f[7]));
  }
}

// kVec: 16-byte accesses to the heads are aligned.
template <typename T, bool kCache, bool kNeighbours, bool kVec>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? (kCache ? 12 : 10) : 8)
    k_head_norm_rotary(const __grid_constant__ RotaryParams p) {
  __shared__ __align__(16) float2 turned[kWarps][kMaxPairs];
  __shared__ __align__(16) float most[kCache ? kWarps : 1][kCache ? 64 : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lanes = p.lanes, at_once = p.at_once, head_of = lane / lanes, s = lane - head_of * lanes;
  const int64_t unit = int64_t(blockIdx.x) * kWarps + warp;
  grid_wait();
  if (unit >= p.tokens * p.slices) return;
  const int64_t token = p.slices == 1 ? unit : unit / p.slices;
  const int32_t first = int32_t(unit - token * p.slices) * p.per_slice;
  const int32_t rotated = p.rows[0].steps + p.rows[1].steps;
  const int32_t end = min(first + p.per_slice, kCache ? rotated + p.rows[2].steps : rotated);

  // this lane's chunks
  const int eighth = p.pairs >> 3;
  const int chunks = p.dim >> 3;
  int turned_a = s, turned_b = s + (chunks >> 1);
  if (!kNeighbours) {
    turned_b = s + eighth;
    if (s >= eighth) turned_a = 2 * s, turned_b = 2 * s + 1;  // behind the rotated ones: 2 eighth + 2 (s - eighth)
  }
  // chunks that are not rotated
  const bool still_a = turned_a >= 2 * eighth, still_b = turned_b >= 2 * eighth;
  // a block's four chunks are in four neighbouring lanes (of values they always are)
  const bool aligned = kNeighbours || 2 * eighth == chunks;
  const bool lane_in = head_of < at_once;
  const bool by_halves = (lanes & (lanes - 1)) == 0;
  const int64_t slot = kCache ? p.slots[token] : 0;
  const bool held = kCache && slot >= 0 && slot < (p.pages << p.page_shift);
  const int64_t row0 = (((slot >> p.page_shift) * p.kv_heads) << p.page_shift) +  // of head 0
                       (slot & ((int64_t(1) << p.page_shift) - 1));

  // the token's cosines and sines
  if (first < rotated) {
    for (int i = lane; i < p.dim / 2; i += 32) {
      float2 t = make_float2(1.0f, 0.0f);  // behind the pairs nothing turns
      if (i < p.pairs) {
        const int32_t ax = p.axis == nullptr ? 0 : min(max(p.axis[i], 0), p.axes - 1);
        t = turn_to_cos_sin(uint64_t(int64_t(p.positions[token * p.axes + ax])) * uint64_t(p.turns[i]));
      }
      turned[warp][i] = t;
    }
    __syncwarp();
  }

  int32_t behind = 0;  // steps of the kinds before
#pragma unroll
  for (int kind = 0; kind < (kCache ? 3 : 2); ++kind) {  // unrolled, so that its fields are constants
    const Rows& r = p.rows[kind];
    const int32_t from = max(first - behind, 0), to = min(end - behind, r.steps);
    behind += r.steps;
    if (from >= to) continue;
    const int ca = kind < 2 ? turned_a : s, cb = kind < 2 ? turned_b : s + (chunks >> 1);
    const bool whole = kind == 2 || aligned;
    int32_t head = from * at_once + head_of;
    const T* src = static_cast<const T*>(r.x) + token * r.st + head * r.sh;
    T* dst = static_cast<T*>(r.out) + token * r.o_st + head * r.o_sh;  // not used on the way into the cache
    // Loads of kAhead heads of 16 bits are under way, each in registers of its own: they
    // are not moved, which would wait for them, hence the unrolled loop.
    constexpr int kAhead = sizeof(T) == 2 && !kCache ? 2 : 1;
    Chunk8<T> raw_a[kAhead] = {}, raw_b[kAhead] = {};
    auto fetch = [&](int32_t at, int u) {
      if (lane_in && at < r.heads)
        raw_a[u] = load_chunk<T, kVec>(src + 8 * ca), raw_b[u] = load_chunk<T, kVec>(src + 8 * cb);
      src += r.step;
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (from + u < to) fetch(head + u * at_once, u);
    // (a, b) -> a (wa cos, wa sin) + b (-wb sin, wb cos)
    uint64_t of_a[8], of_b[8];
    const bool norm = r.weight != nullptr;
    if (!kCache || kind < 2) {
      float w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = 1.0f;
      if (norm && lane_in) {
        auto load = [&](auto vec) {
          constexpr bool kV = decltype(vec)::value;
          if (p.wide_weights) {
            const float* src = static_cast<const float*>(r.weight);
            unpack<float>(load_chunk<float, kV>(src + 8 * ca), w);
            unpack<float>(load_chunk<float, kV>(src + 8 * cb), w + 8);
          } else {
            const T* src = static_cast<const T*>(r.weight);
            unpack<T>(load_chunk<T, kV>(src + 8 * ca), w);
            unpack<T>(load_chunk<T, kV>(src + 8 * cb), w + 8);
          }
        };
        if (p.weight_vec) load(std::true_type{});
        else load(std::false_type{});
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // halves: pair 8 s + j; neighbours: four of each chunk
        const float2 t = turned[warp][kNeighbours ? 4 * (j < 4 ? ca : cb) + (j & 3) : 8 * s + j];
        const float wa = w[kNeighbours ? 2 * j : j], wb = w[kNeighbours ? 2 * j + 1 : 8 + j];
        of_a[j] = pair_of(wa * t.x, wa * t.y), of_b[j] = pair_of(-wb * t.y, wb * t.x);
      }
    }
#pragma unroll 1
    for (int32_t step0 = from; step0 < to; step0 += kAhead)
#pragma unroll
    for (int u = 0; u < kAhead; ++u, head += at_once, dst += r.o_step) {
      const int32_t step = step0 + u;
      if (kAhead > 1 && step >= to) break;
      const bool live = lane_in && head < r.heads;  // the others go along with what they have
      float f[16];
      unpack<T>(raw_a[u], f);
      unpack<T>(raw_b[u], f + 8);
      if (step + kAhead < to) fetch(head + kAhead * at_once, u);
      if (!kCache || kind < 2) {
        if (norm) {
          auto mean = [&]() {
            uint64_t sum2 = 0;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const uint64_t x = pair_of(f[i], f[i + 1]);
              sum2 = fma2(x, x, sum2);
            }
            float sum = unpair(sum2).x + unpair(sum2).y;
            if (by_halves) {
#pragma unroll
              for (int o = 1; o < 16; o <<= 1)
                if (o < lanes) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            } else {
              const float mine = sum;
              sum = 0.0f;
              for (int o = 0; o < lanes; ++o) sum += __shfl_sync(0xFFFFFFFFu, mine, head_of * lanes + o);
            }
            return sum * p.inv_dim;
          };
          float m = mean(), eps = p.eps;
          // squares past the range: 2^-72 of the elements has them within it
          const bool over = __isinff(m);
          if (__any_sync(0xFFFFFFFFu, over)) {
            if (over) {
              eps = 0.0f;
#pragma unroll
              for (int i = 0; i < 16; ++i) f[i] *= 0x1p-72f;
            }
            m = mean();
          }
          const float inv = rsqrtf(m + eps);
          const uint64_t inv2 = pair_of(inv, inv);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float2 x = unpair(mul2(pair_of(f[i], f[i + 1]), inv2));
            f[i] = x.x, f[i + 1] = x.y;
          }
        }
        auto turn = [&](auto part) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float& a = f[kNeighbours ? 2 * j : j];
            float& b = f[kNeighbours ? 2 * j + 1 : 8 + j];
            if (decltype(part)::value && (kNeighbours && j >= 4 ? still_b : still_a)) {
              a *= unpair(of_a[j]).x, b *= unpair(of_b[j]).y;  // an infinity stays in its place
            } else {
              const float2 y = unpair(fma2(pair_of(a, a), of_a[j], mul2(pair_of(b, b), of_b[j])));
              a = y.x, b = y.y;
            }
          }
        };
        if (2 * eighth == chunks) turn(std::false_type{});
        else turn(std::true_type{});
      }
      if (!kCache || kind == 0) {
        if (live) {
          store_chunk<T, kVec>(dst + 8 * ca, f);
          store_chunk<T, kVec>(dst + 8 * cb, f + 8);
        }
        continue;
      }
      if constexpr (kCache) {
        float ma = 0.0f, mb = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ma = max_nan(ma, fabsf(f[i])), mb = max_nan(mb, fabsf(f[8 + i]));
        // the largest of the four chunks of a block
        if (whole) {  // they lie in four neighbouring lanes
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            ma = max_nan(ma, __shfl_xor_sync(0xFFFFFFFFu, ma, o));
            mb = max_nan(mb, __shfl_xor_sync(0xFFFFFFFFu, mb, o));
          }
        } else {
          float* row = most[warp] + head_of * chunks;
          row[ca] = ma, row[cb] = mb;
          __syncwarp();
          const float4 x = *reinterpret_cast<const float4*>(row + (ca & ~3));
          const float4 y = *reinterpret_cast<const float4*>(row + (cb & ~3));
          ma = max_nan(max_nan(x.x, x.y), max_nan(x.z, x.w)), mb = max_nan(max_nan(y.x, y.y), max_nan(y.z, y.w));
          __syncwarp();  // before the next heads' are written
        }
        uint32_t e[2], q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t eb = (__float_as_uint(h ? mb : ma) >> 23) & 0xFFu;
          e[h] = eb == 255u ? 255u : (eb > 2u ? eb - 2u : 0u);
          const float inv = __uint_as_float((254u - min(e[h], 252u)) << 23);
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = f[8 * h + i] * inv;
          q[h] = eb == 255u ? 0u : e2m1x8(y);
        }
        // a head's scales in one word of each of its halves, where they are in order
        uint32_t half_a = e[0], half_b = e[1];
        if (whole && p.dim > 64) {
          half_a |= __shfl_down_sync(0xFFFFFFFFu, half_a, 4) << 8;
          half_b |= __shfl_down_sync(0xFFFFFFFFu, half_b, 4) << 8;
          if (p.dim > 128) {
            half_a |= __shfl_down_sync(0xFFFFFFFFu, half_a, 8) << 16;
            half_b |= __shfl_down_sync(0xFFFFFFFFu, half_b, 8) << 16;
          }
        }
        if (live && held) {
          const int64_t at = row0 + (int64_t(head) << p.page_shift);
          uint8_t* codes = (kind == 1 ? p.k_codes : p.v_codes) + at * (p.dim / 2);
          uint8_t* scales = (kind == 1 ? p.k_scales : p.v_scales) + at * (p.dim / 32);
          *reinterpret_cast<uint32_t*>(codes + ca * 4) = q[0];
          *reinterpret_cast<uint32_t*>(codes + cb * 4) = q[1];
          if (!whole) {
            if ((ca & 3) == 0) scales[ca >> 2] = uint8_t(e[0]);
            if ((cb & 3) == 0) scales[cb >> 2] = uint8_t(e[1]);
          } else if (s == 0) {
            if (p.dim == 64) *reinterpret_cast<uint16_t*>(scales) = uint16_t(half_a | half_b << 8);
            else if (p.dim == 128) *reinterpret_cast<uint32_t*>(scales) = (half_a & 0xFFFFu) | half_b << 16;
            else *reinterpret_cast<uint2*>(scales) = make_uint2(half_a, half_b);
          }
        }
      }
    }
  }
}

// Launches for all tokens.  A warp a token where that fills the GPU (16 warps an
// SM), else a token's steps are dealt over several.
nvfp4_status launch_rotary(RotaryParams& p, int32_t dtype, int32_t weight_dtype, bool cache, bool neighbours, bool vec,
                           cudaStream_t s) {
  int32_t steps = 0;
  for (Rows& r : p.rows) {
    r.steps = (r.heads + p.at_once - 1) / p.at_once;
    r.step = p.at_once * r.sh, r.o_step = p.at_once * r.o_sh;
    steps += r.steps;
  }
  const int64_t want = int64_t(sm_count()) * 16;
  int64_t slices = (want + p.tokens - 1) / p.tokens;
  slices = slices > steps ? steps : slices;
  p.per_slice = int32_t((steps + slices - 1) / slices);
  p.slices = (steps + p.per_slice - 1) / p.per_slice;
  const int64_t blocks = (p.tokens * p.slices + kWarps - 1) / kWarps;
  auto go = [&](auto t) {
    using T = decltype(t);
    auto pick = [&](auto in_cache) {
      constexpr bool kCache = decltype(in_cache)::value;
      return neighbours ? (vec ? k_head_norm_rotary<T, kCache, true, true> : k_head_norm_rotary<T, kCache, true, false>)
                        : (vec ? k_head_norm_rotary<T, kCache, false, true> : k_head_norm_rotary<T, kCache, false, false>);
    };
    void (*kern)(RotaryParams) = pick(std::false_type{});
    if constexpr (sizeof(T) == 2) {
      if (cache) kern = pick(std::true_type{});
    }
    return launch("launch k_head_norm_rotary", kern, dim3(unsigned(blocks)), dim3(kThreads), 0, 0, s, p);
  };
  p.weight_vec = 1;
  for (const Rows& r : p.rows) p.weight_vec = p.weight_vec && aligned16(r.weight);
  p.wide_weights = weight_dtype == MXFP4_FP32 && dtype != MXFP4_FP32;
  if (dtype == MXFP4_FP32) return go(float());
  return dtype == MXFP4_BF16 ? go(__nv_bfloat16()) : go(__half());
}

// What both entry points check of their heads and their rotation; fills `p`.
nvfp4_status check_rotary(const mxfp4_rotary* rotary, int32_t dtype, int32_t weight_dtype, int64_t tokens, int32_t dim,
                          float eps, const std::string& nm, RotaryParams& p) {
  if (!rotary) return fail(NVFP4_EINVAL, nm + ": null pointer");
  if (!mx_dtype_ok(dtype)) return fail(NVFP4_EINVAL, nm + ": unknown element type");
  if (weight_dtype != dtype && weight_dtype != MXFP4_FP32)
    return fail(NVFP4_EINVAL, nm + ": weights must have the heads' type or FP32");
  if (tokens < 0) return fail(NVFP4_EINVAL, nm + ": tokens must not be negative");
  if (tokens > 0x7FFFFFFF) return fail(NVFP4_EUNSUPPORTED, nm + ": too many tokens");
  if (dim < 16 || dim > 256 || dim % 16 != 0)
    return fail(NVFP4_EUNSUPPORTED, nm + ": dim must be a multiple of 16 up to 256");
  if (rotary->pairs < 0 || rotary->pairs % 8 != 0 || rotary->pairs * int64_t(2) > dim)
    return fail(NVFP4_EUNSUPPORTED, nm + ": pairs must be a multiple of 8, and twice as many no more than dim");
  if (rotary->axes < 1 || rotary->axes > 65536) return fail(NVFP4_EINVAL, nm + ": positions need 1 to 65,536 axes");
  if (!(eps >= 1e-12f && eps <= 1.0f)) return fail(NVFP4_EINVAL, nm + ": eps must be from 1e-12 to 1");
  if (tokens > 0 && rotary->pairs > 0 && (!rotary->turns || !rotary->positions))
    return fail(NVFP4_EINVAL, nm + ": null pointer");
  if (reinterpret_cast<uintptr_t>(rotary->turns) % 8 != 0 || reinterpret_cast<uintptr_t>(rotary->axis) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(rotary->positions) % 4 != 0)
    return fail(NVFP4_EALIGN, nm + ": turns, axis and positions must be aligned to their elements");
  p.turns = rotary->turns, p.axis = rotary->axis, p.positions = rotary->positions;
  p.pairs = rotary->pairs, p.axes = rotary->axes;
  p.dim = dim, p.inv_dim = 1.0f / float(dim), p.eps = eps, p.tokens = tokens;
  p.lanes = dim / 16, p.at_once = 32 / p.lanes;
  return NVFP4_OK;
}

nvfp4_status check_rows(const mxfp4_heads* h, int32_t dtype, int32_t weight_dtype, bool out, const std::string& nm,
                        Rows& r, bool& vec) {
  if (!h->x || (out && !h->out)) return fail(NVFP4_EINVAL, nm + ": null pointer");
  const uintptr_t es = uintptr_t(mx_elem_bytes(dtype)), ws = uintptr_t(mx_elem_bytes(weight_dtype));
  if (reinterpret_cast<uintptr_t>(h->x) % es != 0 || reinterpret_cast<uintptr_t>(h->weight) % ws != 0 ||
      (out && reinterpret_cast<uintptr_t>(h->out) % es != 0))
    return fail(NVFP4_EALIGN, nm + ": heads and weights must be aligned to their elements");
  r = {h->x, out ? h->out : nullptr, h->weight, h->st, h->sh, h->o_st, h->o_sh, 0, 0, h->heads, 0};
  const int64_t el = int64_t(16 / es);
  vec = vec && aligned16(h->x) && h->st % el == 0 && h->sh % el == 0;
  if (out) vec = vec && aligned16(h->out) && h->o_st % el == 0 && h->o_sh % el == 0;
  return NVFP4_OK;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status head_norm_rotary(const mxfp4_heads* q, const mxfp4_heads* k, const mxfp4_rotary* rotary,
                                         int32_t dtype, int32_t weight_dtype, int64_t tokens, int32_t dim, float eps,
                                         nvfp4_stream_t stream) {
  const std::string nm("head_norm_rotary");
  RotaryParams p = {};
  nvfp4_status st = check_rotary(rotary, dtype, weight_dtype, tokens, dim, eps, nm, p);
  if (st != NVFP4_OK) return st;
  if (!q) return fail(NVFP4_EINVAL, nm + ": null pointer");
  bool vec = true;
  const mxfp4_heads* both[2] = {q, k};
  for (int i = 0; i < 2; ++i) {
    if (both[i] == nullptr) continue;
    if (both[i]->heads < 1 || both[i]->heads > 65535) return fail(NVFP4_EINVAL, nm + ": 1 to 65,535 heads are needed");
    if (tokens == 0) continue;
    st = check_rows(both[i], dtype, weight_dtype, true, nm, p.rows[i], vec);
    if (st != NVFP4_OK) return st;
  }
  if (tokens == 0) return NVFP4_OK;
  return launch_rotary(p, dtype, weight_dtype, false, rotary->interleaved != 0, vec,
                       reinterpret_cast<cudaStream_t>(stream));
}

extern "C" nvfp4_status mxfp4_cache_write_rotary(const mxfp4_cache* cache, const mxfp4_heads* q, const mxfp4_heads* k,
                                                 const mxfp4_heads* v, const int64_t* slots,
                                                 const mxfp4_rotary* rotary, int32_t dtype, int32_t weight_dtype,
                                                 int64_t tokens, float eps, nvfp4_stream_t stream) {
  const std::string nm("mxfp4_cache_write_rotary");
  int sh = 0;
  nvfp4_status st = check_cache(cache, &sh, nm);
  if (st != NVFP4_OK) return st;
  if (dtype != MXFP4_BF16 && dtype != MXFP4_FP16) return fail(NVFP4_EINVAL, nm + ": heads must be BF16 or FP16");
  RotaryParams p = {};
  st = check_rotary(rotary, dtype, weight_dtype, tokens, cache->dim, eps, nm, p);
  if (st != NVFP4_OK) return st;
  if (!q || !k || !v) return fail(NVFP4_EINVAL, nm + ": null pointer");
  if (q->heads < 1 || q->heads > 65535) return fail(NVFP4_EINVAL, nm + ": 1 to 65,535 query heads are needed");
  if (k->heads != cache->kv_heads || v->heads != cache->kv_heads)
    return fail(NVFP4_EINVAL, nm + ": k and v must have the cache's heads");
  if (v->weight != nullptr) return fail(NVFP4_EINVAL, nm + ": values are not normed");
  if (tokens == 0) return NVFP4_OK;
  if (!slots) return fail(NVFP4_EINVAL, nm + ": null pointer");
  if (reinterpret_cast<uintptr_t>(slots) % 8 != 0)
    return fail(NVFP4_EALIGN, nm + ": slots must be aligned to their elements");
  bool vec = true;
  const mxfp4_heads* all[3] = {q, k, v};
  for (int i = 0; i < 3; ++i) {
    st = check_rows(all[i], dtype, weight_dtype, i == 0, nm, p.rows[i], vec);
    if (st != NVFP4_OK) return st;
  }
  p.slots = slots;
  p.k_codes = static_cast<uint8_t*>(cache->k_codes), p.k_scales = static_cast<uint8_t*>(cache->k_scales);
  p.v_codes = static_cast<uint8_t*>(cache->v_codes), p.v_scales = static_cast<uint8_t*>(cache->v_scales);
  p.pages = cache->pages, p.page_shift = sh, p.kv_heads = cache->kv_heads;
  return launch_rotary(p, dtype, weight_dtype, true, rotary->interleaved != 0, vec,
                       reinterpret_cast<cudaStream_t>(stream));
}
