// Dropout: y = keep x / (1 - p) (+ residual), the mask from philox.hpp and
// never stored; the same call on a gradient is its backward pass. A thread takes
// the eight elements of a run, which are one 16-byte load in bf16 and one call of
// the generator (20 products of 32 x 32 bits, hidden behind the loads). Bound by
// HBM: 4096 x 12288 in bf16 with a residual 55.4 us, 302 MB, 5.4 TB/s.
#include "block_ops.hpp"
#include "philox.hpp"

namespace tp {

namespace {

// Eight elements at p, or the first n of them where the row ends.
template <typename T>
__device__ __forceinline__ void load_run(const T* p, int n, float (&v)[8]) {
  if (n >= 8) {
    load8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.f;
      if (j < n) {
        if constexpr (sizeof(T) == 4)
          v[j] = p[j];
        else
          v[j] = __builtin_bit_cast(float, (uint32_t)p[j] << 16);
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void store_run(T* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    store8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) {
        if constexpr (sizeof(T) == 4)
          p[j] = v[j];
        else
          p[j] = (uint16_t)pack_bf16x2(v[j], 0.f);
      }
  }
}

}  // namespace

template <typename TX, typename TY, bool RES>
__global__ __launch_bounds__(256) void k_dropout(DropoutArgs a) {
  const int64_t runs = (a.k + 7) >> 3, total = a.m * runs;
  const bool drops = a.drop.rng != nullptr;  // NULL: a threshold of 0, which drops nothing and may have no seed
  const PhiloxKey key = drops ? philox_key(a.drop.rng) : PhiloxKey{};
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t run = (int64_t)blockIdx.x * 256 + threadIdx.x; run < total; run += step) {
    int64_t row;
    if (total < ((int64_t)1 << 32))
      row = (uint32_t)run / (uint32_t)runs;
    else
      row = run / runs;
    const int64_t c = (run - row * runs) * 8;
    const int n = (int)min((int64_t)8, a.k - c);
    float x[8], r[8];
    load_run((const TX*)a.x + row * a.ldx + c, n, x);
    if constexpr (RES) load_run((const TY*)a.res + row * a.ldr + c, n, r);
    const u32x4_t w = drops ? philox4x32_10(key, (uint64_t)run) : u32x4_t{};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = philox_drop(w, j, a.drop, x[j]);
      if constexpr (RES) x[j] += r[j];
    }
    store_run((TY*)a.y + row * a.ldy + c, n, x);
  }
}

namespace {

template <typename TX, typename TY>
hipError_t dropout_launch(const DropoutArgs& a, hipStream_t stream) {
  const int64_t total = a.m * ((a.k + 7) >> 3);
  int64_t blocks = (total + 255) / 256;
  if (blocks > 65536) blocks = 65536;  // (threads of a grid in 32 bits; the blocks walk)
  if (a.res != nullptr)
    hipLaunchKernelGGL((k_dropout<TX, TY, true>), dim3((unsigned)blocks), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((k_dropout<TX, TY, false>), dim3((unsigned)blocks), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t stream) {
  if (a.x_bf16)
    return a.y_bf16 ? dropout_launch<uint16_t, uint16_t>(a, stream) : dropout_launch<uint16_t, float>(a, stream);
  return a.y_bf16 ? dropout_launch<float, uint16_t>(a, stream) : dropout_launch<float, float>(a, stream);
}

}  // namespace tp
