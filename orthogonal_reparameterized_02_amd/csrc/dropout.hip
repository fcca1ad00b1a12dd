// Dropout from a counter-based generator, with the residual sum; the mask is
// a function of (seed, element index) and is never stored.  Memory-bound:
// 8191 x 5120 bf16, with residual and back, 73 us for 419 MB = 5.7 TB/s.
#include <algorithm>

#include "attn.h"

namespace poetx {

namespace {

constexpr int NTH = 256;

// Philox 4x32-10 (Salmon et al., 2011): ten rounds of two 32 x 32 -> 64 bit
// products.  One call serves eight elements of 16 random bits each: with 32
// bits an element the products, not the memory, would bound the pass.
__device__ __forceinline__ uint4 philox10(uint32_t c0, uint32_t c1, uint32_t k0, uint32_t k1) {
  uint32_t c2 = 0, c3 = 0;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

template <typename TS> struct alignas(16) Pack8 { TS e[8]; };

// 16-byte loads; NT: non-temporal
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
template <bool NT, typename TS> __device__ __forceinline__ Pack8<TS> load8(const TS* p) {
  constexpr int N = sizeof(Pack8<TS>) / 16;
  const u32x4_t* q = reinterpret_cast<const u32x4_t*>(p);
  u32x4_t t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = NT ? __builtin_nontemporal_load(q + i) : q[i];
  Pack8<TS> v;
  __builtin_memcpy(&v, t, sizeof v);
  return v;
}

// Eight elements a thread.  With a residual both inputs have their last
// reader here and leave the last-level cache to the sum (non-temporal loads:
// forward and backward of 8191 x 5120 bf16 75.3 -> 73 us); the backward
// pass's dy is the residual's gradient too and stays.
template <typename TS, bool RES>
__global__ __launch_bounds__(NTH) void k_dropout(long n, const TS* x, const TS* res, TS* out,
                                                 uint32_t cut, float gain, uint64_t seed,
                                                 uint64_t offset, const uint64_t* offset_dev) {
  const long i = ((long)blockIdx.x * NTH + threadIdx.x) * 8;
  if (i >= n) return;
  if (offset_dev) offset += *offset_dev;
  const uint64_t ctr = (offset + (uint64_t)i) >> 3;
  const uint4 w = philox10((uint32_t)ctr, (uint32_t)(ctr >> 32), (uint32_t)seed, (uint32_t)(seed >> 32));
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
  auto one = [&](int e, float xv, float rv) {
    const uint32_t bits = (e & 1) ? ww[e / 2] >> 16 : ww[e / 2] & 0xffffu;
    const float kept = bits >= cut ? xv * gain : 0.0f;
    return RES ? rv + kept : kept;
  };
  if (i + 8 <= n) {
    using V = Pack8<TS>;
    const V xv = load8<RES>(x + i);
    V rv, yv;
    if constexpr (RES) rv = load8<true>(res + i);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      St<TS>::st(&yv.e[e], one(e, St<TS>::ld(&xv.e[e]), RES ? St<TS>::ld(&rv.e[e]) : 0.0f));
    *reinterpret_cast<V*>(out + i) = yv;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i + e < n)
        St<TS>::st(out + i + e, one(e, St<TS>::ld(x + i + e), RES ? St<TS>::ld(res + i + e) : 0.0f));
  }
}

}  // namespace

template <typename TS>
hipError_t launch_dropout(long n, const TS* x, const TS* res, TS* out, uint32_t cut, uint64_t seed,
                          uint64_t offset, const uint64_t* offset_dev, hipStream_t s) {
  // cut = 65536 drops every element: the gain is never used
  const float gain = cut < 65536u ? 65536.0f / (float)(65536u - cut) : 0.0f;
  constexpr long MOST = 8 * LAUNCH_THREADS;  // elements a launch
  for (; n > 0; n -= MOST, x += MOST, res = res ? res + MOST : nullptr, out += MOST, offset += MOST) {
    const long m = std::min(n, MOST);
    const dim3 grid((unsigned)((m + 8L * NTH - 1) / (8L * NTH)));
    if (res)
      k_dropout<TS, true><<<grid, NTH, 0, s>>>(m, x, res, out, cut, gain, seed, offset, offset_dev);
    else
      k_dropout<TS, false><<<grid, NTH, 0, s>>>(m, x, res, out, cut, gain, seed, offset, offset_dev);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template hipError_t launch_dropout<bf16>(long, const bf16*, const bf16*, bf16*, uint32_t, uint64_t, uint64_t, const uint64_t*, hipStream_t);
template hipError_t launch_dropout<float>(long, const float*, const float*, float*, uint32_t, uint64_t, uint64_t, const uint64_t*, hipStream_t);

}  // namespace poetx
