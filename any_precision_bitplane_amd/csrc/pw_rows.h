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
  static __device__ __forceinline__ floatx8 wide(chunk v) { return __builtin_convertvector(v, floatx8); }
  // one rounding to the row type, to nearest even
  static __device__ __forceinline__ chunk narrow(floatx8 v) { return __builtin_convertvector(v, chunk); }
};

}  // namespace pw
