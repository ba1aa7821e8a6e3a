// Rotation of q and k by position with the append of k and v to the paged
// pools in the same pass; the append into 4-bit pools; and the read-back of
// pool rows.
//
//   (a, b) -> (a cos - b sin, b cos + a sin)         columns paired as pkv_rope says
//   pool[loc] = bf16(y) | e4m3(y * inv) | 4-bit block of y * inv
//
// 4-bit block of 16 columns: S = e4m3(max|y| / 6), code = e2m1(y / S), the
// division as a multiply by the fp32 reciprocal of S. Products and sums of the
// rotation are rounded one by one (no fused multiply-add), so the stored codes
// are those of the same formula in elementary fp32 operations, bit for bit.
//
// Bound by memory: q, k and v are read once, q_out and the pool rows written
// once. One thread owns 16 columns of a head (a whole 4-bit block, 32 bytes of
// bf16) and runs over RPT heads of its token with the angles of those columns
// in registers. 16,384 tokens of 32/8 heads of 128 into bf16 pools: 76.7 us on
// inputs that change from pass to pass, 5,360 GB/s or 0.79 of the copy rate;
// 64 tokens into E4M3 pools: 2.1 us, the launch and the chain of slot, angles
// and rows. Tried and not kept: a persistent grid that takes a token a stage
// through a shared-memory ring by bulk copies (7 % faster at 16,384 tokens than
// this kernel without streaming, slower below 8,000); more threads an SM (82,
// 89 and 113 us at 6, 8 and 10 blocks, where 82 was the default's).
#include <cmath>

#include "pkv_internal.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr long long kStreamBytes = 128ll << 20;  // rows read and written by a launch

enum Rot { kRotNone = 0, kRotHalf = 1, kRotInterleaved = 2 };

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void widen8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}

__device__ __forceinline__ uint4 narrow8(const float* x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 16 scaled values -> 8 code bytes and the block's E4M3 scale byte
__device__ __forceinline__ uint2 quant_fp4(const float* y, uint8_t* scale) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = max_nan(a, fabsf(y[i]));
  const uint16_t s8 = e4m3x2(__fmul_rn(a, 1.0f / 6.0f), 0.f);
  *scale = (uint8_t)(s8 & 0xff);
  const float s = __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(s8) & 0xffffu)));
  const float r = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = __fmul_rn(y[8 * k + i], r);
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(w[k])
        : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]));
  }
  return make_uint2(w[0], w[1]);
}

// 16 bytes of an input row; volatile, so that it stays ahead of the loads whose
// chain it is to overlap. STREAM: read and written once, out of the L2's way.
template <bool STREAM>
__device__ __forceinline__ uint4 load_row(const uint16_t* p) {
  uint4 v;
  if constexpr (STREAM)
    asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  else
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

template <bool STREAM, typename T>
__device__ __forceinline__ void store(T* p, const T& v) {
  if constexpr (STREAM)
    __stcs(p, v);
  else
    *p = v;
}

struct RopeKvArgs {
  const uint16_t *q, *k, *v;  // bf16 rows, token i at i * stride elements
  long long q_stride, k_stride, v_stride;
  uint16_t* q_out;
  void *k_pool, *v_pool;
  const int *loc, *pos;
  const float* cos_sin;
  int max_pos, rotary, first;
  int num_q_heads, num_kv_heads;
  int q_units, kv_units;  // units (RPT heads) of q, and of k or v, in a token
  long long n_threads;
  long long num_slots;
  float k_inv, v_inv;
  int* plan;
};

// Row `head` of width D at a slot (or token): 16 columns (block cb) stored as
// bf16, or scaled and rounded to the pool's codes.
template <int D, bool STREAM>
__device__ __forceinline__ void store_bf16(void* rows, long long slot, int heads, int head, int cb, const uint4& x0,
                                           const uint4& x1) {
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(rows) + (slot * heads + head) * D + cb * 16);
  store<STREAM>(dst, x0);
  store<STREAM>(dst + 1, x1);
}

template <int D, int KV, bool STREAM>
__device__ __forceinline__ void store_coded(void* pool, long long slot, int heads, int head, int cb, const float* x,
                                            float inv) {
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(x[i], inv);
  if constexpr (KV == PKV_KV_FP8_E4M3) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (uint32_t)e4m3x2(y[4 * i], y[4 * i + 1]) | ((uint32_t)e4m3x2(y[4 * i + 2], y[4 * i + 3]) << 16);
    store<STREAM>(reinterpret_cast<uint4*>(static_cast<uint8_t*>(pool) + (slot * heads + head) * D + cb * 16),
                  make_uint4(w[0], w[1], w[2], w[3]));
  } else {
    uint8_t s;
    const uint2 codes = quant_fp4(y, &s);
    uint8_t* tile = static_cast<uint8_t*>(pool) + ((slot / kSegSlots) * heads + head) * fp4_tile_bytes(D);
    const int r = (int)(slot % kSegSlots);
    *reinterpret_cast<uint2*>(tile + r * (D / 2) + cb * 8) = codes;
    tile[kSegSlots * (D / 2) + r * (D / 16) + cb] = s;
  }
}

// The two 8-column vectors of a thread's 16 columns (block cb): whether they are
// rotated, the column of their partners, their first angle, and whether the
// partner's sine counts negative (the first half of the half-split pairing).
template <int ROT>
struct Where {
  int partner[2], angle[2];
  bool rot[2], low[2];
  __device__ __forceinline__ Where(int cb, bool is_v, int first, int rotary) {
    const int half = rotary / 2;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int col = cb * 16 + 8 * v, rel = col - first;
      rot[v] = ROT != kRotNone && !is_v && rel >= 0 && rel < rotary;
      low[v] = rel < half;
      partner[v] = ROT == kRotHalf && rot[v] ? (low[v] ? col + half : col - half) : col;
      angle[v] = ROT == kRotHalf ? (low[v] ? rel : rel - half) : rel / 2;
    }
  }
};

// Cosines and signed sines of those columns.
template <int ROT>
struct Angles {
  float c[16], s[16];
  // row: the position's cosines, then its sines (global or shared memory)
  __device__ __forceinline__ void load(const Where<ROT>& w, const float* row, int half) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      if (!w.rot[v]) continue;
      const float* at = row + w.angle[v];
      if constexpr (ROT == kRotHalf) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 cc = *reinterpret_cast<const float4*>(at + i);
          const float4 ss = *reinterpret_cast<const float4*>(at + half + i);
          const float sg = w.low[v] ? -1.f : 1.f;  // (an exact change of sign)
          c[8 * v + i] = cc.x, c[8 * v + i + 1] = cc.y, c[8 * v + i + 2] = cc.z, c[8 * v + i + 3] = cc.w;
          s[8 * v + i] = sg * ss.x, s[8 * v + i + 1] = sg * ss.y, s[8 * v + i + 2] = sg * ss.z;
          s[8 * v + i + 3] = sg * ss.w;
        }
      } else {
        const float4 cc = *reinterpret_cast<const float4*>(at);
        const float4 ss = *reinterpret_cast<const float4*>(at + half);
        const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          c[8 * v + 2 * i] = c[8 * v + 2 * i + 1] = cv[i];
          s[8 * v + 2 * i] = -sv[i];
          s[8 * v + 2 * i + 1] = sv[i];
        }
      }
    }
  }
  // The rotated columns in fp32 (y) and as bf16 (out; columns that are not
  // rotated keep their bits).
  __device__ __forceinline__ void turn(const Where<ROT>& w, const uint4* own, const uint4* other, float* y,
                                       uint4* out) const {
    float x[16];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      out[v] = own[v];
      widen8(own[v], x + 8 * v);
      float p[8];
      if constexpr (ROT == kRotHalf) {
        widen8(other[v], p);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = x[8 * v + (e ^ 1)];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        y[8 * v + e] = w.rot[v] ? __fadd_rn(__fmul_rn(x[8 * v + e], c[8 * v + e]), __fmul_rn(p[e], s[8 * v + e]))
                                : x[8 * v + e];
      if (w.rot[v]) out[v] = narrow8(y + 8 * v);
    }
  }
};

template <int DK, int DV, int KV, int ROT, int RPT, bool STREAM>
__global__ void __launch_bounds__(kThreads) rope_kv_kernel(RopeKvArgs a) {
  constexpr int CB = DK / 16;  // threads of a unit: 16 columns each
  static_assert(KV == PKV_KV_BF16 || DK == DV, "coded pools: K and V heads of one width");
  pdl_launch_dependents();
  pdl_wait();
  const long long thread = (long long)blockIdx.x * kThreads + threadIdx.x;
  // (threads past the end repeat the last one's loads, for the exchange below)
  const bool idle = thread >= a.n_threads;
  const long long t = idle ? a.n_threads - 1 : thread;
  const int per_token = a.q_units + 2 * a.kv_units;
  const long long unit = t / CB;
  const int cb = (int)(t - unit * CB);
  const long long tok = unit / per_token;
  int u = (int)(unit - tok * per_token);
  const bool is_q = u < a.q_units;
  const bool is_v = u >= a.q_units + a.kv_units;
  if (!is_q) u -= is_v ? a.q_units + a.kv_units : a.q_units;
  const int heads = is_q ? a.num_q_heads : a.num_kv_heads;
  const int h0 = u * RPT, h1 = min(heads, h0 + RPT);
  const bool narrow = is_v && cb * 16 >= DV;  // past the end of a narrower V row
  // The rows are requested first, the token's position and slot after them:
  // the chain position -> angles then runs while the rows are on their way.
  const int width = is_v ? DV : DK;
  const uint16_t* src = (is_q   ? a.q + tok * a.q_stride
                         : is_v ? a.v + tok * a.v_stride
                                : a.k + tok * a.k_stride);
  const int half = a.rotary / 2;
  const Where<ROT> where(cb, is_v, a.first, a.rotary);
  // Partners of the half-split pairing are held by other threads of the row:
  // where a row's threads lie in one warp they hand them over, else they are
  // read a second time (from L1).
  constexpr bool kExchange = ROT == kRotHalf && 32 % CB == 0;
  uint4 own[RPT][2], other[kExchange ? 1 : RPT][2];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const uint16_t* row = src + min(h0 + i, h1 - 1) * width;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      own[i][v] = load_row<STREAM>(row + (narrow ? 0 : cb * 16 + 8 * v));
      if (ROT == kRotHalf && !kExchange) other[i][v] = load_row<STREAM>(row + (narrow ? 0 : where.partner[v]));
    }
  }
  const int pos = ROT != kRotNone ? a.pos[tok] : 0;
  const long long slot = a.loc[tok];
  bool live = !idle && !narrow;  // this thread stores
  if (ROT != kRotNone && (pos < 0 || pos >= a.max_pos)) {
    if (live && cb == 0 && unit == tok * per_token) record_error(a.plan, PKV_DEV_BAD_POSITION, (int)tok);
    live = false;
  } else if (!is_q && (slot < 0 || slot >= a.num_slots)) {
    if (live && cb == 0 && u == 0 && !is_v) record_error(a.plan, PKV_DEV_BAD_SLOT, (int)tok);
    live = false;
  }
  Angles<ROT> angles;
  if (live) angles.load(where, a.cos_sin + (long long)pos * a.rotary, half);
  const bool odd = (half / 8) & 1;  // the partner of one vector is then the other one elsewhere
  const int lane0 = threadIdx.x & 31 & ~(CB - 1);
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int h = h0 + i;
    uint4* partner = other[kExchange ? 0 : i];
    if constexpr (kExchange) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int from = lane0 + (where.partner[v] >> 4);
        const uint4 x = odd ? own[i][v ^ 1] : own[i][v];
        partner[v] = make_uint4(__shfl_sync(0xffffffffu, x.x, from), __shfl_sync(0xffffffffu, x.y, from),
                                __shfl_sync(0xffffffffu, x.z, from), __shfl_sync(0xffffffffu, x.w, from));
      }
    }
    if (!live || h >= h1) continue;
    float y[16];
    uint4 out[2];
    angles.turn(where, own[i], partner, y, out);
    if (is_q) {
      store_bf16<DK, STREAM>(a.q_out, tok, heads, h, cb, out[0], out[1]);
    } else if constexpr (KV == PKV_KV_BF16) {
      if (is_v)
        store_bf16<DV, STREAM>(a.v_pool, slot, heads, h, cb, out[0], out[1]);
      else
        store_bf16<DK, STREAM>(a.k_pool, slot, heads, h, cb, out[0], out[1]);
    } else {
      store_coded<DK, KV, STREAM>(is_v ? a.v_pool : a.k_pool, slot, heads, h, cb, y, is_v ? a.v_inv : a.k_inv);
    }
  }
}

template <int DK, int DV, int KV, int ROT>
int run_rope(RopeKvArgs& a, int n, cudaStream_t st) {
  // One head a thread while the launch is small (latency), four once there are
  // enough threads to fill the GPU (16,384 tokens of 32/8 heads of 128: 95 us
  // with one, 79 with two or four). Past the L2's size the rows stream (same
  // tokens, inputs that change: 81.9 us without, 76.7 with loads and stores
  // streaming, neither alone gains; below it the attention that follows finds q
  // in the L2).
  const long long rows = (long long)n * (a.num_q_heads + 2 * a.num_kv_heads);
  const int rpt = rows * (DK / 16) >= (1 << 19) ? 4 : 1;
  const bool stream = rows * DK * 4 > kStreamBytes;
  a.q_units = a.q ? (a.num_q_heads + rpt - 1) / rpt : 0;
  a.kv_units = (a.num_kv_heads + rpt - 1) / rpt;
  a.n_threads = (long long)n * (a.q_units + 2 * a.kv_units) * (DK / 16);
  const long long blocks = (a.n_threads + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffll) return PKV_ERR_UNSUPPORTED;
  auto kernel = rpt == 1 ? rope_kv_kernel<DK, DV, KV, ROT, 1, false>
                : stream ? rope_kv_kernel<DK, DV, KV, ROT, 4, true>
                         : rope_kv_kernel<DK, DV, KV, ROT, 4, false>;
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, st, a) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <int ROT>
int dispatch_rope(const pkv_config& cfg, RopeKvArgs& a, int n, cudaStream_t st) {
  if (cfg.kv_dtype == PKV_KV_FP4_E2M1) return run_rope<128, 128, PKV_KV_FP4_E2M1, ROT>(a, n, st);
  if constexpr (ROT != kRotNone) {
    if (cfg.kv_dtype == PKV_KV_FP8_E4M3) return run_rope<128, 128, PKV_KV_FP8_E4M3, ROT>(a, n, st);
    if (cfg.head_dim == 128) return run_rope<128, 128, PKV_KV_BF16, ROT>(a, n, st);
    if (cfg.head_dim == 64) return run_rope<64, 64, PKV_KV_BF16, ROT>(a, n, st);
    if (cfg.head_dim == 192) return run_rope<192, 128, PKV_KV_BF16, ROT>(a, n, st);
  }
  return PKV_ERR_UNSUPPORTED;
}

// ---------------------------------------------------------------- read-back
// One thread reads 8 columns of a K and of a V row and writes each as one
// 16-byte vector, so that neighbouring threads fill whole lines.
struct GetKvArgs {
  const void *k_pool, *v_pool;
  uint16_t *k, *v;
  const int* loc;
  int heads, dk, dv;
  long long n_threads, num_slots;
  float k_scale, v_scale;
  int* plan;
};

template <int KV>
__global__ void __launch_bounds__(256) get_kv_kernel(GetKvArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const long long t = (long long)blockIdx.x * 256 + threadIdx.x;
  if (t >= a.n_threads) return;
  const int vecs = a.dk / 8;
  const long long row = t / vecs;
  const int c = (int)(t - row * vecs) * 8;  // first column
  const long long tok = row / a.heads;
  const int h = (int)(row - tok * a.heads);
  const long long slot = a.loc[tok];
  if (slot < 0 || slot >= a.num_slots) {
    if (h == 0 && c == 0) record_error(a.plan, PKV_DEV_BAD_SLOT, (int)tok);
    return;
  }
  // both rows' codes first
  uint4 x[2];
  uint32_t scale8[2] = {0, 0};
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const int d = which ? a.dv : a.dk;
    if (c >= d) continue;
    const uint8_t* pool = static_cast<const uint8_t*>(which ? a.v_pool : a.k_pool);
    if constexpr (KV == PKV_KV_BF16) {
      x[which] = *reinterpret_cast<const uint4*>(pool + ((slot * a.heads + h) * d + c) * 2);
    } else if constexpr (KV == PKV_KV_FP8_E4M3) {
      const uint2 y = *reinterpret_cast<const uint2*>(pool + (slot * a.heads + h) * d + c);
      x[which].x = y.x, x[which].y = y.y;
    } else {
      const uint8_t* tile = pool + ((slot / kSegSlots) * a.heads + h) * fp4_tile_bytes(d);
      const int r = (int)(slot % kSegSlots);
      x[which].x = *reinterpret_cast<const uint32_t*>(tile + r * (d / 2) + c / 2);
      scale8[which] = tile[kSegSlots * (d / 2) + r * (d / 16) + c / 16];
    }
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const int d = which ? a.dv : a.dk;
    if (c >= d) continue;
    const float scale = which ? a.v_scale : a.k_scale;
    uint4* dst = reinterpret_cast<uint4*>((which ? a.v : a.k) + (tok * a.heads + h) * d + c);
    if constexpr (KV == PKV_KV_BF16) {
      *dst = x[which];
    } else {
      uint32_t w[4];  // 8 values as f16 pairs, exact
      if constexpr (KV == PKV_KV_FP8_E4M3) {
        w[0] = e4m3x2_to_f16x2((uint16_t)(x[which].x & 0xffffu));
        w[1] = e4m3x2_to_f16x2((uint16_t)(x[which].x >> 16));
        w[2] = e4m3x2_to_f16x2((uint16_t)(x[which].y & 0xffffu));
        w[3] = e4m3x2_to_f16x2((uint16_t)(x[which].y >> 16));
      } else {
        const uint32_t s2 = e4m3x2_to_f16x2((uint16_t)(scale8[which] | (scale8[which] << 8)));
        e2m1x8_to_f16x2(x[which].x, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = mul_f16x2(w[i], s2);  // exact: at most 6 significant bits
      }
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = __half2float(__ushort_as_half((unsigned short)(w[i] & 0xffffu)));
        const float hi = __half2float(__ushort_as_half((unsigned short)(w[i] >> 16)));
        o[i] = pack_bf16(__fmul_rn(lo, scale), __fmul_rn(hi, scale));
      }
      *dst = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

}  // namespace

int launch_rope_set_kv(Ctx& c, const pkv_rope* rope, void* k_pool, void* v_pool, const int32_t* loc,
                       const int32_t* pos, const void* q, long long q_stride, const void* k, long long k_stride,
                       const void* v, long long v_stride, void* q_out, int n, float k_inv, float v_inv,
                       cudaStream_t st) {
  RopeKvArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.loc = loc;
  a.pos = pos;
  a.cos_sin = rope ? rope->d_cos_sin : nullptr;
  a.max_pos = rope ? rope->max_positions : 0;
  a.rotary = rope ? rope->rotary_dim : 0;
  a.first = rope ? rope->rotary_offset : 0;
  a.num_q_heads = q ? c.cfg.num_q_heads : 0;
  a.num_kv_heads = c.cfg.num_kv_heads;
  a.num_slots = (long long)c.cfg.num_pages * c.cfg.page_size;
  a.k_inv = k_inv;
  a.v_inv = v_inv;
  a.plan = make_meta(c).plan;
  if (!rope) return dispatch_rope<kRotNone>(c.cfg, a, n, st);
  return rope->interleaved ? dispatch_rope<kRotInterleaved>(c.cfg, a, n, st)
                           : dispatch_rope<kRotHalf>(c.cfg, a, n, st);
}

int launch_get_kv_buffer(Ctx& c, const void* k_pool, const void* v_pool, const int32_t* loc, void* k, void* v, int n,
                         float k_scale, float v_scale, cudaStream_t st) {
  GetKvArgs a;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.k = static_cast<uint16_t*>(k);
  a.v = static_cast<uint16_t*>(v);
  a.loc = loc;
  a.heads = c.cfg.num_kv_heads;
  a.dk = c.cfg.head_dim;  // the K heads are at least as wide as the V heads (check_config)
  a.dv = head_dim_v(c.cfg);
  a.n_threads = (long long)n * a.heads * (a.dk / 8);
  a.num_slots = (long long)c.cfg.num_pages * c.cfg.page_size;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.plan = make_meta(c).plan;
  const long long blocks = (a.n_threads + 255) / 256;
  if (blocks > 0x7fffffffll) return PKV_ERR_UNSUPPORTED;
  auto kernel = c.cfg.kv_dtype == PKV_KV_BF16       ? get_kv_kernel<PKV_KV_BF16>
                : c.cfg.kv_dtype == PKV_KV_FP8_E4M3 ? get_kv_kernel<PKV_KV_FP8_E4M3>
                                                    : get_kv_kernel<PKV_KV_FP4_E2M1>;
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(256), 0, st, a) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
