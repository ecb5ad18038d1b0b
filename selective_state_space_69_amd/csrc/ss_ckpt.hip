// Activation checkpoints in 8 bits for gfx950: blocks of 32 channels share a
// power-of-two unit and hold signed 8-bit multiples of it (what a backward pass
// needs is recomputed or kept: "A Survey of Mamba" summary, hardware-aware
// computation).
//
//   e = max(1, E - 6), E the biased exponent of the block's largest |x|
//   q = clamp(round(x 2^(127 - e)), +-127),  x ~ q 2^(e - 127)
//
// Both scalings are exact, so packing rounds once (to the integer) and unpacking
// not at all; 2^(127 - e) and 2^(e - 127) are formed in the exponent field.
// Streaming kernels: a thread takes 8 channels (16-byte bf16 loads, 8-byte
// stores of q), the four threads of a block of 32 exchange its largest |x| by
// two lane swaps within their quad.  Bound by memory: 16384 x 5120 bf16 packs in 48
// us and unpacks in 40 (5.3 and 6.3 TB/s of the least traffic; a large copy: 5.1).
#include "ss_device.hpp"

namespace ss {
namespace {

constexpr int kVec = 8;
constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = int64_t(1) << 22;   // a grid's threads stay below 2^32

struct CkptParams {
  const void* x;
  void* out;
  const int8_t* q;
  int8_t* qo;
  const uint8_t* e;
  uint8_t* eo;
  int64_t total;      // threads' vectors: rows * 4 * ceil(D / 32)
  int64_t xs;
  int32_t D, nq;      // nq = vectors of a row, 4 ceil(D / 32)
};

// bits of the largest |x| of the quad's 32 values (NaN above infinity)
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  uint32_t o = uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0xB1, 0xf, 0xf, true));
  m = m > o ? m : o;
  o = uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x4E, 0xf, 0xf, true));
  return m > o ? m : o;
}

// VEC: D a multiple of 8 and every row 16-byte aligned
template <typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void pack_kernel(CkptParams p) {
  // whole quads run together: total is a multiple of 4
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < p.total;
       i += int64_t(gridDim.x) * kThreads) {
    const int64_t row = p.total <= INT32_MAX ? int64_t(uint32_t(i) / uint32_t(p.nq)) : i / p.nq;
    const int v = int(i - row * p.nq), c = v * kVec;
    const T* x = static_cast<const T*>(p.x) + row * p.xs + c;
    float f[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) f[j] = 0.0f;
    if constexpr (VEC) {
      if (c < p.D) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 w = unpack4(load_raw4(x + 4 * h));
          f[4 * h] = w.x; f[4 * h + 1] = w.y; f[4 * h + 2] = w.z; f[4 * h + 3] = w.w;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (c + j < p.D) f[j] = to_f32(x[j]);
    }
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const uint32_t b = __float_as_uint(f[j]) & 0x7fffffffu;
      m = m > b ? m : b;
    }
    const uint32_t E = quad_max(m) >> 23;
    const uint32_t e = E == 255u ? 255u : (E > 7u ? E - 6u : 1u);
    const float up = __uint_as_float((254u - (e == 255u ? 254u : e)) << 23);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const float r = __builtin_fminf(__builtin_fmaxf(__builtin_rintf(f[j] * up), -127.0f), 127.0f);
      const int qi = e == 255u ? 0 : int(r);
      w[j / 4] |= uint32_t(qi & 255) << (8 * (j % 4));
    }
    int8_t* q = p.qo + row * p.D + c;
    if constexpr (VEC) {
      if (c < p.D) *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (c + j < p.D) q[j] = int8_t(w[j / 4] >> (8 * (j % 4)));
    }
    if ((v & 3) == 0) p.eo[row * (p.nq / 4) + v / 4] = uint8_t(e);
  }
}

template <typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void unpack_kernel(CkptParams p) {
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < p.total;
       i += int64_t(gridDim.x) * kThreads) {
    const int64_t row = p.total <= INT32_MAX ? int64_t(uint32_t(i) / uint32_t(p.nq)) : i / p.nq;
    const int v = int(i - row * p.nq), c = v * kVec;
    if (c >= p.D) continue;
    const uint32_t e = p.e[row * (p.nq / 4) + v / 4];
    const float unit = e == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(e << 23);
    const int8_t* q = p.q + row * p.D + c;
    T* x = static_cast<T*>(p.out) + row * p.xs + c;
    float f[kVec];
    if constexpr (VEC) {
      const uint2 r = *reinterpret_cast<const uint2*>(q);
      const uint32_t w[2] = {r.x, r.y};
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        f[j] = float(int8_t(w[j / 4] >> (8 * (j % 4)))) * unit;
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(x) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(x + 4) = make_float4(f[4], f[5], f[6], f[7]);
      } else {
        uint32_t o[4];
#pragma unroll
        for (int h = 0; h < 4; ++h)
          o[h] = uint32_t(f32_to_bf16(f[2 * h])) | (uint32_t(f32_to_bf16(f[2 * h + 1])) << 16);
        *reinterpret_cast<uint4*>(x) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (c + j < p.D) store_out<T>(x + j, float(q[j]) * unit);
    }
  }
}

bool vec_ok(const ss_ckpt_desc_t& d, const void* x) {
  const int64_t xs = d.x_stride ? d.x_stride : d.dim;
  return d.dim % kVec == 0 && xs % kVec == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
}

CkptParams params(const ss_ckpt_desc_t& d, unsigned* blocks) {
  CkptParams p{};
  p.D = int32_t(d.dim);
  p.nq = int32_t((d.dim + 31) / 32 * 4);
  p.xs = d.x_stride ? d.x_stride : d.dim;
  p.total = d.rows * p.nq;
  const int64_t b = (p.total + kThreads - 1) / kThreads;
  *blocks = unsigned(b < kMaxBlocks ? b : kMaxBlocks);
  return p;
}

}  // namespace

int launch_ckpt_pack(const ss_ckpt_desc_t& d, const void* x, int8_t* q, uint8_t* e,
                     void* stream) {
  unsigned blocks;
  CkptParams p = params(d, &blocks);
  p.x = x;
  p.qo = q;
  p.eo = e;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool vec = vec_ok(d, x);
  if (d.dtype == SS_BF16) {
    if (vec) pack_kernel<uint16_t, true><<<blocks, kThreads, 0, st>>>(p);
    else pack_kernel<uint16_t, false><<<blocks, kThreads, 0, st>>>(p);
  } else {
    if (vec) pack_kernel<float, true><<<blocks, kThreads, 0, st>>>(p);
    else pack_kernel<float, false><<<blocks, kThreads, 0, st>>>(p);
  }
  return int(hipGetLastError());
}

int launch_ckpt_unpack(const ss_ckpt_desc_t& d, const int8_t* q, const uint8_t* e, void* x,
                       void* stream) {
  unsigned blocks;
  CkptParams p = params(d, &blocks);
  p.q = q;
  p.e = e;
  p.out = x;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool vec = vec_ok(d, x);
  if (d.dtype == SS_BF16) {
    if (vec) unpack_kernel<uint16_t, true><<<blocks, kThreads, 0, st>>>(p);
    else unpack_kernel<uint16_t, false><<<blocks, kThreads, 0, st>>>(p);
  } else {
    if (vec) unpack_kernel<float, true><<<blocks, kThreads, 0, st>>>(p);
    else unpack_kernel<float, false><<<blocks, kThreads, 0, st>>>(p);
  }
  return int(hipGetLastError());
}

}  // namespace ss
