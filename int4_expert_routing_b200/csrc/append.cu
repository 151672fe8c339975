// Appending keys and values to the paged cache, with each head's RMSNorm and
// the rotary positions applied on the way (flint_kv_append).
//
// Memory bound: every row is read once and written once.  A warp has one token
// (or, in a short call, some of its heads), so that nothing waits for another
// warp.  A head of D elements belongs to D / 16 neighbouring lanes; a lane
// holds two 8-element chunks (16-byte loads), chosen so that both partners of
// every rotated pair are in the same lane: chunks l and l + rope_dim / 16 for
// the half-split pairing, any two for the interleaved one.  So the rotation
// needs no exchange, the norm one reduction over D / 16 lanes, and a lane's
// eight angles are those of all heads and stay in registers.  16,384 tokens of
// 32 + 4 heads of 128 (335 MB): 60 us, 5.6 TB/s (5.4 with its launch, of 6.5 of a copy), with two passes loaded ahead
// of the two at work; 68 without, 77 with five at once (fewer warps fit), 108
// with blocks of tokens that wait for their angles.
//
// turn = pos * f in fp64 with f = theta^(-2i/rope_dim) / 2 pi from the host,
// its fraction (exact to 2^-53 of the product) to fp32, then sincospi; a lane
// does two of the token's 64 and the lanes exchange them.  fp32 angles would be
// off by 2^-24 of pos, which is a whole radian at a position of 10^7.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace flint {

constexpr int kApThreads = 128;
constexpr int kApWarps = kApThreads / 32;
constexpr int kApFillWarps = 148 * 16;  // warps that keep the memory busy
constexpr int kApUnroll = 2;   // passes loaded while as many are worked on

struct AppendKArgs {
  AppendArgs a;
  double freq[64];  // turns per position
};

FLINT_DEV void unpack8(const uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
FLINT_DEV uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// eight values over `scale` as E4M3, to nearest, saturating
FLINT_DEV uint2 pack8_e4m3(const float (&x)[8], float scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unsigned short h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(h)
        : "f"(__fdiv_rn(x[2 * i + 1], scale)), "f"(__fdiv_rn(x[2 * i], scale)));
    w[i] = h;
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// `parts` warps share a token's heads
template <int kD>
__global__ void __launch_bounds__(kApThreads)
    k_kv_append(const __grid_constant__ AppendKArgs p, int parts) {
  constexpr int kLanes = kD / 16;      // lanes of a head
  constexpr int kHeads = 32 / kLanes;  // heads of a pass
  const AppendArgs &a = p.a;
  const int lane = threadIdx.x & 31, l = lane % kLanes, grp = lane / kLanes;
  const int item = blockIdx.x * kApWarps + (threadIdx.x >> 5);
  const int t = item / parts, part = item - t * parts;
  const int heads = a.q_heads + 2 * a.heads;
  const int passes = (heads + kHeads - 1) / kHeads;
  const int first = passes * part / parts, last = passes * (part + 1) / parts;
  const int h = a.rope_dim / 16;  // chunk pairs that turn
  const bool turns = l < h;
  // this lane's chunks
  const bool split = !a.interleaved && turns;
  const int ca = split ? l : 2 * l, cb = split ? l + h : 2 * l + 1;

  pdl_wait();
  pdl_trigger();
  if (t >= a.T) return;
  const int64_t slot = a.slots[t];
  const int pos = a.pos[t];
  auto row_of = [&](int hd) {
    return hd < a.q_heads ? a.q + (int64_t)t * a.q_stride + hd * kD
           : hd < a.q_heads + a.heads
               ? a.k + (int64_t)t * a.k_stride + (hd - a.q_heads) * kD
               : a.v + (int64_t)t * a.v_stride + (hd - a.q_heads - a.heads) * kD;
  };
  uint4 va[kApUnroll], vb[kApUnroll], na[kApUnroll], nb[kApUnroll];
  auto load = [&](int base, uint4 (&va)[kApUnroll], uint4 (&vb)[kApUnroll]) {
#pragma unroll
    for (int u = 0; u < kApUnroll; ++u) {
      const int hd = (base + u) * kHeads + grp;
      if (base + u < last && hd < heads) {
        const uint16_t *src = row_of(hd);
        va[u] = *reinterpret_cast<const uint4 *>(src + 8 * ca);
        vb[u] = *reinterpret_cast<const uint4 *>(src + 8 * cb);
      }
    }
  };
  load(first, va, vb);
  long long off = -1;
  if (slot >= 0) {
    const int64_t page = slot / a.page_size;
    if (page < a.num_pages)
      off = page * a.page_stride + (slot - page * a.page_size) * a.token_stride;
    else
      set_status(a.status, kStatusDevice);
  }
  if (off < 0) return;
  float2 cs[8];  // cos and sin of angles 8 l + j
  if (h > 0) {
    float c[kD / 64], s[kD / 64];
#pragma unroll
    for (int i = 0; i < kD / 64; ++i) {
      const double turn = (double)pos * p.freq[32 * i + lane];
      sincospif(2.f * (float)(turn - rint(turn)), &s[i], &c[i]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int from = (8 * l + j) & 31;
      cs[j] = make_float2(__shfl_sync(0xffffffffu, c[0], from), __shfl_sync(0xffffffffu, s[0], from));
      if (kD == 128) {
        const float2 hi = make_float2(__shfl_sync(0xffffffffu, c[kD / 64 - 1], from),
                                      __shfl_sync(0xffffffffu, s[kD / 64 - 1], from));
        if (l >= 4) cs[j] = hi;
      }
    }
  }
  for (int base = first; base < last; base += kApUnroll) {
    load(base + kApUnroll, na, nb);
#pragma unroll
    for (int u = 0; u < kApUnroll; ++u) {
      if (base + u >= last) break;
      const int hd = (base + u) * kHeads + grp;
      const bool is_q = hd < a.q_heads, is_v = hd >= a.q_heads + a.heads;
      float xa[8], xb[8];
      unpack8(va[u], xa);
      unpack8(vb[u], xb);
      const uint16_t *norm = is_q ? a.q_norm : a.k_norm;
      // the lanes of a head take the same branches; the shuffles stay inside it
      if (a.q_norm || a.k_norm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += xa[j] * xa[j] + xb[j] * xb[j];
#pragma unroll
        for (int o = 1; o < kLanes; o *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (!is_v && norm) {
          const float r = rsqrtf(ss * (1.f / kD) + (float)FLINT_RMS_EPS);
          float wa[8], wb[8];
          unpack8(*reinterpret_cast<const uint4 *>(norm + 8 * ca), wa);
          unpack8(*reinterpret_cast<const uint4 *>(norm + 8 * cb), wb);
#pragma unroll
          for (int j = 0; j < 8; ++j) xa[j] *= r * wa[j], xb[j] *= r * wb[j];
        }
      }
      if (hd >= heads) continue;
      if (!is_v && turns) {
        if (!a.interleaved) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = xa[j], y = xb[j];
            xa[j] = x * cs[j].x - y * cs[j].y;
            xb[j] = y * cs[j].x + x * cs[j].y;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 e = cs[j + 4];
            float x = xa[2 * j], y = xa[2 * j + 1];
            xa[2 * j] = x * cs[j].x - y * cs[j].y;
            xa[2 * j + 1] = y * cs[j].x + x * cs[j].y;
            x = xb[2 * j], y = xb[2 * j + 1];
            xb[2 * j] = x * e.x - y * e.y;
            xb[2 * j + 1] = y * e.x + x * e.y;
          }
        }
      }
      if (is_q) {
        uint16_t *dst = a.q_out + (int64_t)t * a.q_out_stride + hd * kD;
        *reinterpret_cast<uint4 *>(dst + 8 * ca) = pack8(xa);
        *reinterpret_cast<uint4 *>(dst + 8 * cb) = pack8(xb);
      } else {
        const int kh = is_v ? hd - a.q_heads - a.heads : hd - a.q_heads;
        const long long e = off + kh * (long long)a.head_stride;
        if (a.type == FLINT_KV_BF16) {
          uint16_t *dst = reinterpret_cast<uint16_t *>(is_v ? a.vc : a.kc) + e;
          *reinterpret_cast<uint4 *>(dst + 8 * ca) = pack8(xa);
          *reinterpret_cast<uint4 *>(dst + 8 * cb) = pack8(xb);
        } else {
          const float *scales = is_v ? a.v_scale : a.k_scale;
          const float s = scales ? scales[kh] : 1.f;
          uint8_t *dst = reinterpret_cast<uint8_t *>(is_v ? a.vc : a.kc) + e;
          *reinterpret_cast<uint2 *>(dst + 8 * ca) = pack8_e4m3(xa, s);
          *reinterpret_cast<uint2 *>(dst + 8 * cb) = pack8_e4m3(xb, s);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kApUnroll; ++u) va[u] = na[u], vb[u] = nb[u];
  }
}

cudaError_t launch_append(const AppendArgs &a, double theta, cudaStream_t st) {
  AppendKArgs p;
  p.a = a;
  // theta^(-2i / rope_dim) from its powers at the bits of i, and those as roots
  // of the largest (a root halves an error): one call of pow instead of 64
  // (2 us), six roundings instead of one
  p.freq[0] = 1.0 / 6.283185307179586476925;
  int top = 1;
  while (4 * top < a.rope_dim) top *= 2;
  double f[7];
  f[6] = pow(theta, -2.0 * top / (a.rope_dim > 0 ? a.rope_dim : 1));
  int at = 6;
  for (int bit = top; bit > 1; bit /= 2, --at) f[at - 1] = sqrt(f[at]);
  for (int bit = 1; bit <= top; bit *= 2, ++at)
    for (int i = bit; i < 2 * bit; ++i) p.freq[i] = p.freq[i - bit] * f[at];
  // A token's heads go to one warp, or in a call of few tokens to several, one
  // pass each at the least.
  const int per_pass = 512 / a.head_dim, heads = a.q_heads + 2 * a.heads;
  const int passes = (heads + per_pass - 1) / per_pass;
  int parts = kApFillWarps / a.T;
  parts = parts < 1 ? 1 : parts > passes ? passes : parts;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)a.T * parts + kApWarps - 1) / kApWarps));
  cfg.blockDim = dim3(kApThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_step("kv append launch");
  return a.head_dim == 128 ? cudaLaunchKernelEx(&cfg, k_kv_append<128>, p, parts)
                           : cudaLaunchKernelEx(&cfg, k_kv_append<64>, p, parts);
}

}  // namespace flint
