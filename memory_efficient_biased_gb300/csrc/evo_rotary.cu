// evo_rotary.cu — rotary positions (include/evo_seq.h): queries and keys in one launch.
//
// Mathematics.  The angle of token t and pair i, in turns, is positions[t] · inv_freq[i] / 2π.  The
// frequency's part of a turn is kept as a 64-bit fraction F = round(2^64 frac(inv_freq / 2π)), and the
// product position · F, taken modulo 2^64, is the angle modulo a turn with no rounding of its own, however
// far the position.  Its upper 32 bits as a signed fraction of half a turn go through sincospif.  (An
// angle formed in 32 bits would be off by 0.06 at a position of 10^6.)
//
// Work.  A thread keeps one token and VEC pairs, whose sines and cosines it forms once, and takes
// every heads_apart-th head of q and then of k: its loads and stores are VEC elements wide, and a
// head's threads lie next to each other.  Features that pass are copied by threads behind all of
// these (in the same warps, the two paths one behind the other, a half turned head took twice the time).  F is formed once a block, in shared memory, as its few operations in 64 bits are
// the dearest here (a GB300 issues two a clock and SM).
//
// Bound by the bytes: every element read and written once.  16,384 tokens of 40 heads of 128 take 54 us, 6.2 TB/s; 6,092 of 40
// with half of the head turned 19.6, 6.4 TB/s.  Inputs are read with an evict-first hint, so that the outputs are what stays in L2
// for the attention (57 and 25 us without; on the stores too it gained nothing).
#include <cmath>

#include "evo_seq_check.h"

namespace evo {
namespace {

struct RotaryArgs {
  const uint16_t *q, *k;
  uint16_t *q_out, *k_out;
  long long q_stride, k_stride, q_out_stride, k_out_stride;
  const int* positions;
  const double* inv_freq;
  int tokens, q_heads, heads, D, half;  // heads: of q and k together
  int pairs, passing;                   // threads a head: for its pairs, and (not in place) for the features that pass
  int heads_apart;                      // threads a token and unit
  long long turning;                    // threads that turn pairs; those behind them copy
  float factor, sine;                   // sine: ±factor
};

constexpr int kRotaryThreads = 256, kMaxPairs = 64;

template <int VEC>
struct Pack;
template <>
struct Pack<8> { using T = uint4; };
template <>
struct Pack<4> { using T = uint2; };
template <>
struct Pack<2> { using T = uint32_t; };
template <>
struct Pack<1> { using T = uint16_t; };

template <bool BF16, int N>
__device__ __forceinline__ void unpack_row(const typename Pack<N>::T& v, float (&x)[N]) {
  union {
    typename Pack<N>::T v;
    uint16_t e[N];
  } u;
  u.v = v;
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = to_f32<BF16>(u.e[i]);
}
template <bool BF16, int N>
__device__ __forceinline__ typename Pack<N>::T pack_row(const float (&x)[N]) {
  union {
    typename Pack<N>::T v;
    uint32_t w[(N + 1) / 2];
    uint16_t e[N];
  } u;
  if constexpr (N == 1) {
    u.e[0] = static_cast<uint16_t>(pack2<BF16>(x[0], 0.0f));
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) u.w[i] = pack2<BF16>(x[2 * i], x[2 * i + 1]);
  }
  return u.v;
}

constexpr int kAtOnce = 4;  // heads of a thread whose loads are under way together (the outputs may be the inputs: left to
                            // the compiler, each head's loads waited for the stores of the one before)

// VEC pairs a thread: their first and second features are VEC next to each other each (halves), or
// 2 VEC next to each other, in turns (INTERLEAVED; two loads where VEC is 8).
template <bool BF16, bool INTERLEAVED, int VEC>
__global__ void __launch_bounds__(kRotaryThreads) evo_rotary_kernel(const __grid_constant__ RotaryArgs a) {
  __shared__ unsigned long long turn[kMaxPairs];
  for (int i = threadIdx.x; i < a.half; i += kRotaryThreads) {
    const double x = a.inv_freq[i] * 0.15915494309189533577;  // 1 / 2π
    // (a fraction that rounds to 1 saturates in the conversion, 2^-64 turns off)
    turn[i] = static_cast<unsigned long long>((x - floor(x)) * 18446744073709551616.0);
  }
  __syncthreads();
  long long id = static_cast<long long>(blockIdx.x) * kRotaryThreads + threadIdx.x;
  const bool copy = id >= a.turning;
  if (copy) id -= a.turning;
  if (copy && a.passing == 0) return;
  const int units = copy ? a.passing : a.pairs;
  const long long rest = id / units;
  const int unit = static_cast<int>(id - rest * units);
  const long long t = rest / a.heads_apart;
  if (t >= a.tokens) return;
  const int first = static_cast<int>(rest - t * a.heads_apart);
  auto in = [&](int h) {
    return h < a.q_heads ? a.q + t * a.q_stride + h * a.D : a.k + t * a.k_stride + (h - a.q_heads) * a.D;
  };
  auto out = [&](int h) {
    return h < a.q_heads ? a.q_out + t * a.q_out_stride + h * a.D : a.k_out + t * a.k_out_stride + (h - a.q_heads) * a.D;
  };
  using T = typename Pack<VEC>::T;
  if (copy) {
    const int at = 2 * a.half + unit * VEC;
    for (int h0 = first; h0 < a.heads; h0 += 2 * kAtOnce * a.heads_apart) {
      T x[2 * kAtOnce];
#pragma unroll
      for (int e = 0; e < 2 * kAtOnce; ++e)
        if (const int h = h0 + e * a.heads_apart; h < a.heads) x[e] = __ldcs(reinterpret_cast<const T*>(in(h) + at));
#pragma unroll
      for (int e = 0; e < 2 * kAtOnce; ++e)
        if (const int h = h0 + e * a.heads_apart; h < a.heads) *reinterpret_cast<T*>(out(h) + at) = x[e];
    }
    return;
  }
  float c[VEC], s[VEC];
  const long long pos = a.positions[t];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const unsigned long long angle = static_cast<unsigned long long>(pos) * turn[unit * VEC + i];
    sincospif(static_cast<float>(static_cast<int>(angle >> 32)) * 0x1p-31f, &s[i], &c[i]);
    s[i] *= a.sine;
    c[i] *= a.factor;
  }
  const int at = INTERLEAVED ? 2 * unit * VEC : unit * VEC, gap = INTERLEAVED ? VEC : a.half;
  for (int h0 = first; h0 < a.heads; h0 += kAtOnce * a.heads_apart) {
    T lo[kAtOnce], hi[kAtOnce];
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e)
      if (const int h = h0 + e * a.heads_apart; h < a.heads) {
        lo[e] = __ldcs(reinterpret_cast<const T*>(in(h) + at));
        hi[e] = __ldcs(reinterpret_cast<const T*>(in(h) + at + gap));
      }
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) {
      const int h = h0 + e * a.heads_apart;
      if (h >= a.heads) break;
      float x[VEC], y[VEC];
      unpack_row<BF16, VEC>(lo[e], x);
      unpack_row<BF16, VEC>(hi[e], y);
      if constexpr (!INTERLEAVED || VEC == 1) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float u = x[i], v = y[i];
          x[i] = fmaf(u, c[i], -v * s[i]);
          y[i] = fmaf(v, c[i], u * s[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {  // pair i: elements 2i and 2i + 1 of x and y together
          float(&z)[VEC] = i < VEC / 2 ? x : y;
          const int p = 2 * i % VEC;
          const float u = z[p], v = z[p + 1];
          z[p] = fmaf(u, c[i], -v * s[i]);
          z[p + 1] = fmaf(v, c[i], u * s[i]);
        }
      }
      uint16_t* to = out(h) + at;
      *reinterpret_cast<T*>(to) = pack_row<BF16, VEC>(x);
      *reinterpret_cast<T*>(to + gap) = pack_row<BF16, VEC>(y);
    }
  }
}

template <bool BF16, bool INTERLEAVED, int VEC>
cudaError_t launch_rotary_t(const RotaryArgs& a, cudaStream_t st) {
  const long long threads = a.turning + static_cast<long long>(a.tokens) * a.passing * a.heads_apart;
  evo_rotary_kernel<BF16, INTERLEAVED, VEC>
      <<<static_cast<unsigned>((threads + kRotaryThreads - 1) / kRotaryThreads), kRotaryThreads, 0, st>>>(a);
  return cudaGetLastError();
}
template <bool BF16, bool INTERLEAVED>
cudaError_t launch_rotary_v(const RotaryArgs& a, int vec, cudaStream_t st) {
  return vec == 8   ? launch_rotary_t<BF16, INTERLEAVED, 8>(a, st)
         : vec == 4 ? launch_rotary_t<BF16, INTERLEAVED, 4>(a, st)
         : vec == 2 ? launch_rotary_t<BF16, INTERLEAVED, 2>(a, st)
                    : launch_rotary_t<BF16, INTERLEAVED, 1>(a, st);
}

}  // namespace
}  // namespace evo

using namespace evo;

extern "C" evo_status_t evo_rotary(const void* q, const void* k, const int32_t* positions, const double* inv_freq,
                                   void* q_out, void* k_out, evo_seq_shape_t shape, const evo_rotary_t* rotary,
                                   evo_dtype_t dtype, const evo_seq_strides_t* strides, void* stream) {
  if (!rotary) return EVO_ERR_NULL_POINTER;
  if (rotary->flags & ~(EVO_ROTARY_INTERLEAVED | EVO_ROTARY_INVERSE) || !std::isfinite(rotary->factor))
    return EVO_ERR_BAD_ARGUMENT;
  if ((k == nullptr) != (k_out == nullptr)) return EVO_ERR_BAD_ARGUMENT;
  if (dtype != EVO_F16 && dtype != EVO_BF16) return EVO_ERR_BAD_DTYPE;
  const int64_t T = shape.tokens, Hq = shape.q_heads, Hk = k ? shape.kv_heads : 0, D = shape.head_dim, R = rotary->rotary_dim;
  if (T < 0 || T > (int64_t(1) << 31) - 1024 || Hq < 1 || Hq > 65535 || Hk < 0 || Hk > 16384 || D < 8 || D > 128 || D % 8 ||
      R < 2 || R > D || R % 2)
    return EVO_ERR_BAD_SHAPE;
  RotaryArgs a{};
  if (!stride_ok(strides ? strides->q : 0, Hq * D, &a.q_stride) || !stride_ok(strides ? strides->k : 0, Hk * D, &a.k_stride) ||
      !stride_ok(rotary->q_out, Hq * D, &a.q_out_stride) || !stride_ok(rotary->k_out, Hk * D, &a.k_out_stride))
    return EVO_ERR_BAD_LAYOUT;
  if (T == 0) return EVO_OK;
  if (!q || !q_out || !positions || !inv_freq) return EVO_ERR_NULL_POINTER;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(positions, 4) ||
      !aligned(inv_freq, 8))
    return EVO_ERR_MISALIGNED;
  const bool q_self = q == q_out && a.q_stride == a.q_out_stride, k_self = k && k == k_out && a.k_stride == a.k_out_stride;
  const Span in[] = {q_self ? flat(nullptr, 0) : strided(q, T, a.q_stride, Hq * D),
                     k_self ? flat(nullptr, 0) : strided(k, T, a.k_stride, Hk * D), flat(positions, size_t(T) * 4),
                     flat(inv_freq, size_t(R) * 4)};
  const Span outs[] = {strided(q_out, T, a.q_out_stride, Hq * D), strided(k_out, T, a.k_out_stride, Hk * D)};
  if (aliased(in, outs)) return EVO_ERR_ALIASING;
  int sms = 0;
  int* fallback = nullptr;
  const evo_status_t ds = host_device(&sms, &fallback);
  if (ds != EVO_OK) return ds;
  a.q = static_cast<const uint16_t*>(q), a.k = static_cast<const uint16_t*>(k);
  a.q_out = static_cast<uint16_t*>(q_out), a.k_out = static_cast<uint16_t*>(k_out);
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.tokens = static_cast<int>(T);
  a.q_heads = static_cast<int>(Hq);
  a.heads = static_cast<int>(Hq + Hk);
  a.D = static_cast<int>(D);
  a.half = static_cast<int>(R / 2);
  a.factor = rotary->factor == 0.0f ? 1.0f : rotary->factor;
  a.sine = rotary->flags & EVO_ROTARY_INVERSE ? -a.factor : a.factor;
  const bool bf16 = dtype == EVO_BF16, inter = rotary->flags & EVO_ROTARY_INTERLEAVED;
  // the widest accesses that the pairs allow (rows and heads start on 16 bytes)
  const int vec = a.half % 8 == 0 ? 8 : a.half % 4 == 0 ? 4 : a.half % 2 == 0 ? 2 : 1;
  const bool in_place = q_self && (!k || k_self);
  a.pairs = a.half / vec;
  a.passing = in_place ? 0 : (a.D - 2 * a.half) / vec;
  // A thread takes about ten heads, for the cost of its sines, while there are enough threads to fill the SMs.
  const int64_t fill = int64_t(sms) * 2048, per = T * (a.pairs + a.passing);
  int64_t apart = (a.heads + 9) / 10;
  if (per * apart < fill) apart = (fill + per - 1) / per;
  a.heads_apart = static_cast<int>(apart < a.heads ? apart : a.heads);
  a.turning = T * a.pairs * a.heads_apart;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = bf16 ? (inter ? launch_rotary_v<true, true>(a, vec, st) : launch_rotary_v<true, false>(a, vec, st))
                             : (inter ? launch_rotary_v<false, true>(a, vec, st) : launch_rotary_v<false, false>(a, vec, st));
  return e == cudaSuccess ? EVO_OK : cuda_fail("rotary launch", e);
}
