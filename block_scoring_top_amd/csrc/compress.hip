// compress.hip - key compression and store, the step just upstream of the
// scorer.
//
// Page "Qwen3.8-Flash-Next Day-0 in SGLang", QSA section: the indexer has one
// shared key head; each run of 4 raw index keys becomes one compressed key by
// an FP32 average, a normalisation and a rotation with the MRoPE position of
// the run's first token, stored as bf16 at the page-aligned full_slot/4; the
// raw keys of a request's unfinished block are held in a 4-slot ring instead
// of a full-context raw-key cache.
//
// Readings: the average is ((k0 + k1) + k2) + k3 in FP32 times 0.25; the
// normalisation is division by the L2 norm (a zero mean stays zero); the
// rotation pairs dims (i, i + rot/2) over the first rot dims (rotate-half),
// pair i turning by P * theta^(-2i/rot) where P is the t, h or w component of
// the block's MRoPE position chosen by contiguous sections.  The ring's final
// state is that of writing every new token at slot p mod 4 in position order.
//
// One wavefront per compressed key (blockIdx.y = request, blockIdx.x = the
// request's n-th completed block).  The work is a short dependent chain, so
// every global load is issued up front.  Lanes load the 4 raw keys as
// 16-byte chunks into LDS, then own dims (lane, lane + 64): FP32 mean, a
// wave-wide max and sum of squares (scaled by the max so that neither
// overflows nor underflows), angles reduced in FP64 and turned into FP32
// sin/cos, FP32 rotation, one rounding to bf16, and a coalesced 256-byte
// store.  The first wave of each request also updates its ring, after it has
// consumed any ring entries.
//
// A ring of 4 slots holds what a request that only grows needs.  One that is cut
// back (rejected draft tokens) needs the unfinished block of where it is cut, which
// later tokens at the same positions mod 4 have overwritten there; a ring of S
// slots, the token at position p in slot p mod S, still has it after a cut by S - 3.
#include <cmath>
#include <type_traits>

#include "idx4.h"
#include "kernels.h"

namespace bs {

namespace {

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t h) { return __uint_as_float(h << 16); }

// FP32 -> bf16 bit pattern, round to nearest, ties to even; NaN -> quiet NaN.
__device__ __forceinline__ uint32_t f32_to_bf16_rne(float x) {
  const uint32_t u = __float_as_uint(x);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0x7FC0u;
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

template <class T>
__device__ __forceinline__ T wave_sum(T v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

__device__ __forceinline__ float wave_max(float v) {
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

}  // namespace

// FOUR: the keys, rounded to bf16 all the same, are then quantised into the
// 4-bit cache (kcache: codes) in place of being stored as they are.  Half a step of
// a 4-bit value is a quarter of it, so that a key on the wrong side of a tie would
// be far off: norm and rotation are in FP64 then (8,192 tokens: 5.0 us, 4.7 in FP32).
// DEEP: the ring has more than 4 slots (with their number known 8,192 tokens take 3.9
// and 4.4 us, 4.0 and 4.5 without).
template <bool FOUR, bool DEEP>
__global__ __launch_bounds__(64) void compress_kernel(
    const uint16_t* __restrict__ k_raw, int32_t num_tok, const int32_t* __restrict__ req_tok_ptr,
    const int32_t* __restrict__ tok_start, const int32_t* __restrict__ mrope_pos, int32_t max_tok,
    int32_t rot, int32_t sec0, int32_t sec01, double base,
    uint16_t* ring, int32_t* ring_pos, int32_t deep_slots,
    const int32_t* __restrict__ page_table, int32_t pt_stride,
    uint16_t* __restrict__ kcache, uint8_t* __restrict__ scales, int64_t num_pages) {
  __shared__ __align__(16) uint16_t raw[4][kDim];
  typedef std::conditional_t<FOUR, double, float> real;
  __shared__ real ys[kDim];
  __shared__ __align__(16) uint16_t outs[kDim];

  const int b = blockIdx.y, item = blockIdx.x, lane = threadIdx.x;
  const int tp = req_tok_ptr[b];
  const int64_t s = tok_start[b];
  const int n = min(req_tok_ptr[b + 1] - tp, max_tok);
  if (s < 0 || n <= 0) return;
  const int64_t e = s + n - 1;                  // last new position
  const int64_t j0 = s >> 2;                    // block of the first new token
  const int64_t nb = ((e + 1) >> 2) - j0;       // blocks completed by this call
  if (item >= (nb > 1 ? nb : 1)) return;
  // k_raw row of new position p >= s, clamped into the buffer
  auto row_of = [&](int64_t p) -> int64_t {
    const int64_t t = tp + (p - s);
    return t < 0 ? 0 : (t >= num_tok ? num_tok - 1 : t);
  };
  const int u = lane >> 4, c16 = lane & 15;     // raw key u, 16-byte chunk c16

  // The slots of a position's raw key and of its block's MRoPE position (a
  // power of two of each).
  const int ring_slots = DEEP ? deep_slots : 4, slot_mask = ring_slots - 1, block_mask = slot_mask >> 2;
  auto ring_key = [&](int64_t p) { return ring + ((int64_t)b * ring_slots + ((int)p & slot_mask)) * kDim; };
  auto ring_block = [&](int64_t p) {
    return ring_pos + ((int64_t)b * (ring_slots >> 2) + ((int)(p >> 2) & block_mask)) * 3;
  };

  // Ring update of the request's first wave: lanes u write the newest token
  // p <= e with p mod 4 == u, when that token is new, and those before it that a
  // deeper ring still holds.  Its loads read k_raw only and the first are issued
  // first; its stores come last.
  const int64_t pu = e - ((e - u) & 3);
  const bool ring_slot = item == 0 && pu >= s;
  uint4 ring_val = make_uint4(0, 0, 0, 0);
  if (ring_slot) ring_val = reinterpret_cast<const uint4*>(k_raw + row_of(pu) * kDim)[c16];

  if (item < nb) {
    const int64_t j = j0 + item;
    const int64_t p = 4 * j + u;
    const uint16_t* src = p >= s ? k_raw + row_of(p) * kDim : ring_key(p);
    const uint4 v = reinterpret_cast<const uint4*>(src)[c16];
    const int64_t lp = (4 * j) >> 6;            // logical page of the block
    const int page = lp < pt_stride ? page_table[(int64_t)b * pt_stride + lp] : -1;
    int P[3];
    const int64_t pf = 4 * j;                   // the block's first token
    if (mrope_pos == nullptr) {
      P[0] = P[1] = P[2] = (int)pf;
    } else {
      const int32_t* mp = pf >= s ? mrope_pos + row_of(pf) * 3 : ring_block(pf);
      P[0] = mp[0];
      P[1] = mp[1];
      P[2] = mp[2];
    }
    reinterpret_cast<uint4*>(&raw[u][0])[c16] = v;

    // Rotation of the pairs of this lane's dims (lane, lane + 64), in
    // revolutions: frequency base^i with base = theta^(-2/rot) (squarings in
    // FP64), angle P * base^i / (2 pi) reduced exactly to [-1/2, 1/2] in
    // FP64, then sin and cos of pi * 2f in FP32.
    const int half = rot >> 1;
    real cs[2], sn[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int d = lane + 64 * h;
      cs[h] = 1;
      sn[h] = 0;
      if (d < rot) {
        const int i = d < half ? d : d - half;
        const int comp = i < sec0 ? 0 : (i < sec01 ? 1 : 2);
        double f = 1.0, bb = base;
#pragma unroll
        for (int bit = 0; bit < 6; ++bit) {
          if ((i >> bit) & 1) f *= bb;
          bb *= bb;
        }
        const double rev = (double)P[comp] * f * 0.15915494309189535;  // 1 / (2 pi)
        if constexpr (FOUR) {
          sincospi(2.0 * (rev - rint(rev)), &sn[h], &cs[h]);
        } else {
          const float fr = (float)(rev - rint(rev));
          sincospif(2.f * fr, &sn[h], &cs[h]);
        }
      }
    }
    __syncthreads();

    float m[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int d = lane + 64 * h;
      float acc = bf16_bits_to_f32(raw[0][d]);
      acc += bf16_bits_to_f32(raw[1][d]);
      acc += bf16_bits_to_f32(raw[2][d]);
      acc += bf16_bits_to_f32(raw[3][d]);
      m[h] = acc * 0.25f;
    }
    real y0 = 0, y1 = 0;
    if constexpr (FOUR) {  // squares of FP32 values stay in range
      const double m0 = m[0], m1 = m[1], sum = wave_sum(m0 * m0 + m1 * m1);
      const double r = sum < INFINITY ? 1.0 / sqrt(sum) : __builtin_nan("");
      if (sum != 0) y0 = m0 * r, y1 = m1 * r;
    } else {
      const float amax = wave_max(fmaxf(fabsf(m[0]), fabsf(m[1])));
      if (amax > 0.f) {
        const float a0 = m[0] / amax, a1 = m[1] / amax;
        const float r = 1.0f / sqrtf(wave_sum(a0 * a0 + a1 * a1));
        y0 = a0 * r;
        y1 = a1 * r;
      }
    }
    ys[lane] = y0;
    ys[lane + 64] = y1;
    __syncthreads();

#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int d = lane + 64 * h;
      real out = ys[d];
      if (d < rot) out = d < half ? ys[d] * cs[h] - ys[d + half] * sn[h] : ys[d] * cs[h] + ys[d - half] * sn[h];
      outs[d] = (uint16_t)f32_to_bf16_rne((float)out);
    }
    __syncthreads();

    if (page >= 0 && page < num_pages) {
      const int64_t slot = (int64_t)page * (kPage / 4) + (j & (kPage / 4 - 1));
      if constexpr (FOUR) {
        if (lane < kDim / 8) {
          Chunk<Bf16> x;
          x.load(outs + lane * 8);
          bool bad;
          const uint32_t ex = group_exponent(quad_max(x.top()), bad);
          reinterpret_cast<uint32_t*>(kcache)[slot * (kIdxCodes / 4) + lane] = bad ? 0u : x.codes(kv4_scale(ex));
          if ((lane & 3) == 0) scales[slot * kIdxScales + lane / 4] = (uint8_t)(bad ? kExpNan : ex);
        }
      } else {
        reinterpret_cast<uint32_t*>(kcache + slot * kDim)[lane] = reinterpret_cast<const uint32_t*>(outs)[lane];
      }
    }
  }

  if (item == 0) {
    // The block above read its ring entries into LDS before its first
    // barrier, so these stores come after those reads.
    if (ring_slot) reinterpret_cast<uint4*>(ring_key(pu))[c16] = ring_val;
    if constexpr (DEEP)
      for (int64_t p = pu - 4; p >= s && p > e - ring_slots; p -= 4)
        reinterpret_cast<uint4*>(ring_key(p))[c16] = reinterpret_cast<const uint4*>(k_raw + row_of(p) * kDim)[c16];
    const int64_t p0 = e - (e & 3);             // newest block start <= e
    if (ring_pos != nullptr && lane < 3)
      for (int64_t p = p0; p >= s && p > p0 - ring_slots; p -= 4)
        ring_block(p)[lane] = mrope_pos != nullptr ? mrope_pos[row_of(p) * 3 + lane] : (int32_t)p;
  }
}

namespace {

template <bool FOUR>
int launch(const uint16_t* k_raw, int32_t num_tok, const int32_t* req_tok_ptr, const int32_t* tok_start,
           const int32_t* mrope_pos, int32_t num_req, int32_t max_tok, int32_t rotary_dim, int32_t sec_t, int32_t sec_h,
           double theta, uint16_t* ring, int32_t* ring_pos, int32_t ring_slots, const int32_t* page_table, int32_t pt_stride,
           uint16_t* kcache, uint8_t* scales, int64_t num_pages, hipStream_t stream) {
  const int items = max(1, (max_tok + 3) / 4);
  // theta^(-2/rot), the ratio of successive pair frequencies
  const double base = rotary_dim > 0 ? std::pow(theta, -2.0 / (double)rotary_dim) : 1.0;
  auto go = [&](auto deep) {
    hipLaunchKernelGGL((compress_kernel<FOUR, decltype(deep)::value>), dim3(items, num_req), dim3(64), 0, stream, k_raw,
                       num_tok, req_tok_ptr, tok_start, mrope_pos, max_tok, rotary_dim, sec_t, sec_t + sec_h, base, ring,
                       ring_pos, ring_slots, page_table, pt_stride, kcache, scales, num_pages);
  };
  if (ring_slots > 4)
    go(std::true_type());
  else
    go(std::false_type());
  return hipGetLastError() == hipSuccess ? BS_OK : BS_ERR_LAUNCH;
}

}  // namespace

int launch_compress(const uint16_t* k_raw, int32_t num_tok, const int32_t* req_tok_ptr, const int32_t* tok_start,
                    const int32_t* mrope_pos, int32_t num_req, int32_t max_tok, int32_t rotary_dim,
                    int32_t sec_t, int32_t sec_h, double theta, uint16_t* ring, int32_t* ring_pos, int32_t ring_slots,
                    const int32_t* page_table, int32_t pt_stride, uint16_t* kcache, int64_t num_pages,
                    hipStream_t stream) {
  return launch<false>(k_raw, num_tok, req_tok_ptr, tok_start, mrope_pos, num_req, max_tok, rotary_dim, sec_t, sec_h,
                       theta, ring, ring_pos, ring_slots, page_table, pt_stride, kcache, nullptr, num_pages, stream);
}

int launch_compress4(const uint16_t* k_raw, int32_t num_tok, const int32_t* req_tok_ptr, const int32_t* tok_start,
                     const int32_t* mrope_pos, int32_t num_req, int32_t max_tok, int32_t rotary_dim,
                     int32_t sec_t, int32_t sec_h, double theta, uint16_t* ring, int32_t* ring_pos, int32_t ring_slots,
                     const int32_t* page_table, int32_t pt_stride, uint8_t* codes, uint8_t* scales, int64_t num_pages,
                     hipStream_t stream) {
  return launch<true>(k_raw, num_tok, req_tok_ptr, tok_start, mrope_pos, num_req, max_tok, rotary_dim, sec_t, sec_h,
                      theta, ring, ring_pos, ring_slots, page_table, pt_stride, reinterpret_cast<uint16_t*>(codes), scales, num_pages,
                      stream);
}

}  // namespace bs
