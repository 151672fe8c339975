// Appending keys and values to the paged cache, with each head's RMSNorm and
// the rotary positions applied on the way (flint_kv_append).
//
// Memory bound: every row is read once and written once.  A head of D
// elements belongs to D / 16 neighbouring lanes; a lane holds two 8-element
// chunks (16-byte loads), chosen so that both partners of every rotated pair
// are in the same lane: chunks l and l + rope_dim / 16 for the half-split
// pairing, any two for the interleaved one.  So the rotation needs no
// exchange and the norm one reduction over D / 16 lanes.
//
// The angles of a token are computed once for its block: turn = pos * f in
// fp64 with f = theta^(-2i/rope_dim) / 2 pi from the host, its fraction (exact
// to 2^-53 of the product) to fp32, then sincospi.  fp32 angles would be off
// by 2^-24 of pos, which is a whole radian at a position of 10^7.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace flint {

constexpr int kApThreads = 256;
constexpr int kApUnroll = 4;   // heads a lane group loads ahead of using them
constexpr int kApMaxTok = 4;   // tokens of a block

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

// kD head size; kTok tokens a block
template <int kD, int kTok>
__global__ void __launch_bounds__(kApThreads)
    k_kv_append(const __grid_constant__ AppendKArgs p) {
  constexpr int kLanes = kD / 16;                // lanes of a head
  constexpr int kGroups = kApThreads / kLanes;   // heads in flight a block
  __shared__ float2 cs[kTok][64];  // angle i = 8 l + j at [8 j + l]: lanes read neighbours
  __shared__ long long at[kTok];   // the token's element offset in the cache, -1: skip
  const AppendArgs &a = p.a;
  const int tid = threadIdx.x, l = tid % kLanes, grp = tid / kLanes;
  const int t0 = blockIdx.x * kTok, nt = min(kTok, a.T - t0);
  const int heads = a.q_heads + 2 * a.heads;
  const int h = a.rope_dim / 16;  // chunk pairs that turn
  int ca, cb;                     // this lane's chunks
  if (!a.interleaved) {
    ca = l < h ? l : 2 * l;
    cb = l < h ? l + h : 2 * l + 1;
  } else {
    ca = 2 * l, cb = 2 * l + 1;
  }
  const bool turns = l < h;

  pdl_wait();
  pdl_trigger();
  if (tid < nt) {
    const int64_t slot = a.slots[t0 + tid];
    long long off = -1;
    if (slot >= 0) {
      const int64_t page = slot / a.page_size;
      if (page < a.num_pages)
        off = page * a.page_stride + (slot - page * a.page_size) * a.token_stride;
      else
        set_status(a.status, kStatusDevice);
    }
    at[tid] = off;
  }
  for (int i = tid; i < nt * (a.rope_dim / 2); i += kApThreads) {
    const int t = i / (a.rope_dim / 2), f = i % (a.rope_dim / 2);
    const double turn = (double)a.pos[t0 + t] * p.freq[f];
    float s, c;
    sincospif(2.f * (float)(turn - rint(turn)), &s, &c);
    cs[t][8 * (f & 7) + (f >> 3)] = make_float2(c, s);
  }

  for (int base = 0; base < nt * heads; base += kGroups * kApUnroll) {
    uint4 va[kApUnroll], vb[kApUnroll];
#pragma unroll
    for (int u = 0; u < kApUnroll; ++u) {
      const int item = base + u * kGroups + grp;
      if (item < nt * heads) {
        const int t = item / heads, hd = item % heads;
        const uint16_t *src =
            hd < a.q_heads ? a.q + (int64_t)(t0 + t) * a.q_stride + hd * kD
            : hd < a.q_heads + a.heads
                ? a.k + (int64_t)(t0 + t) * a.k_stride + (hd - a.q_heads) * kD
                : a.v + (int64_t)(t0 + t) * a.v_stride + (hd - a.q_heads - a.heads) * kD;
        va[u] = *reinterpret_cast<const uint4 *>(src + 8 * ca);
        vb[u] = *reinterpret_cast<const uint4 *>(src + 8 * cb);
      }
    }
    if (base == 0) __syncthreads();
#pragma unroll
    for (int u = 0; u < kApUnroll; ++u) {
      const int item = base + u * kGroups + grp;
      const bool in = item < nt * heads;
      const int t = in ? item / heads : 0, hd = in ? item % heads : 0;
      const bool is_q = hd < a.q_heads, is_v = hd >= a.q_heads + a.heads;
      const long long off = at[t];
      float xa[8], xb[8];
      unpack8(va[u], xa);
      unpack8(vb[u], xb);
      const uint16_t *norm = is_q ? a.q_norm : a.k_norm;
      // the lanes of a head take the same branches; the shuffles stay inside it
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += xa[j] * xa[j] + xb[j] * xb[j];
#pragma unroll
      for (int o = 1; o < kLanes; o *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (!in || off < 0) continue;
      if (!is_v) {
        if (norm) {
          const float r = rsqrtf(ss * (1.f / kD) + (float)FLINT_RMS_EPS);
          float wa[8], wb[8];
          unpack8(*reinterpret_cast<const uint4 *>(norm + 8 * ca), wa);
          unpack8(*reinterpret_cast<const uint4 *>(norm + 8 * cb), wb);
#pragma unroll
          for (int j = 0; j < 8; ++j) xa[j] *= r * wa[j], xb[j] *= r * wb[j];
        }
        if (turns) {
          if (!a.interleaved) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 c = cs[t][8 * j + l];
              const float x = xa[j], y = xb[j];
              xa[j] = x * c.x - y * c.y;
              xb[j] = y * c.x + x * c.y;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 c = cs[t][8 * j + l], e = cs[t][8 * (j + 4) + l];
              float x = xa[2 * j], y = xa[2 * j + 1];
              xa[2 * j] = x * c.x - y * c.y;
              xa[2 * j + 1] = y * c.x + x * c.y;
              x = xb[2 * j], y = xb[2 * j + 1];
              xb[2 * j] = x * e.x - y * e.y;
              xb[2 * j + 1] = y * e.x + x * e.y;
            }
          }
        }
      }
      if (is_q) {
        uint16_t *dst = a.q_out + (int64_t)(t0 + t) * a.q_out_stride + hd * kD;
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
  }
}

cudaError_t launch_append(const AppendArgs &a, double theta, cudaStream_t st) {
  AppendKArgs p;
  p.a = a;
  // theta^(-2i / rope_dim) from its powers at the bits of i: seven calls of pow
  // instead of 64 (2 us), six roundings instead of one
  p.freq[0] = 1.0 / 6.283185307179586476925;
  for (int bit = 1; 2 * bit < a.rope_dim; bit *= 2) {
    const double f = pow(theta, -2.0 * bit / a.rope_dim);
    for (int i = bit; i < 2 * bit && i < 64; ++i) p.freq[i] = p.freq[i - bit] * f;
  }
  // Blocks of one token spread a short call over more SMs; blocks of four
  // share the angles' latency and keep more loads in flight.
  const bool many = a.T >= 4 * 148 * 4;
  const int tok = many ? kApMaxTok : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.T + tok - 1) / tok);
  cfg.blockDim = dim3(kApThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_step("kv append launch");
  if (a.head_dim == 128)
    return many ? cudaLaunchKernelEx(&cfg, k_kv_append<128, kApMaxTok>, p)
                : cudaLaunchKernelEx(&cfg, k_kv_append<128, 1>, p);
  return many ? cudaLaunchKernelEx(&cfg, k_kv_append<64, kApMaxTok>, p)
              : cudaLaunchKernelEx(&cfg, k_kv_append<64, 1>, p);
}

}  // namespace flint
