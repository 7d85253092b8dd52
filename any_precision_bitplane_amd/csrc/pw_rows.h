// Row access of the operators around the layer: rows of H elements (fp32, fp16
// or bf16) in chunks of eight, computed in fp32.
#pragma once

#include "pw_device.h"
#include "pw_internal.h"

namespace pw {

typedef float floatx8 __attribute__((ext_vector_type(8)));

template <int DT>
struct RowType;
template <>
struct RowType<PW_F32> { using elem = float; };
template <>
struct RowType<PW_F16> { using elem = _Float16; };
template <>
struct RowType<PW_BF16> { using elem = __bf16; };

// Eight consecutive elements; rows start on 16-byte boundaries, so fp32 chunks
// are two 16-byte accesses.
template <int DT>
struct Row {
  using elem = typename RowType<DT>::elem;
  typedef elem chunk __attribute__((ext_vector_type(8), aligned(16)));

  static __device__ __forceinline__ chunk load(const elem* p) { return *reinterpret_cast<const chunk*>(p); }
  static __device__ __forceinline__ void store(elem* p, chunk v) { *reinterpret_cast<chunk*>(p) = v; }
  // The same past the L2s, for what is used once.  16-bit outputs stored so took
  // the norm's fp16 [4096][4096] from 24.5 to 21.0 us, its gradient's from 30.6
  // to 28.5 and unpermute's T = 4096, H = 4096, k = 2 from 20.4 to 17.6, and cost
  // nothing at a few rows; fp32 ones were slower (the gradient's [16384][4096]
  // 192 -> 207), so they are stored as usual.
  static __device__ __forceinline__ chunk load_once(const elem* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const chunk*>(p));
  }
  static __device__ __forceinline__ void store_once(elem* p, chunk v) {
    if constexpr (DT == PW_F32) store(p, v);
    else __builtin_nontemporal_store(v, reinterpret_cast<chunk*>(p));
  }
  static __device__ __forceinline__ floatx8 wide(chunk v) { return __builtin_convertvector(v, floatx8); }
  // one rounding to the row type, to nearest even
  static __device__ __forceinline__ chunk narrow(floatx8 v) { return __builtin_convertvector(v, chunk); }
};

}  // namespace pw
