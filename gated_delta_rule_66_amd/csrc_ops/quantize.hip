// quantize.hip -- rows to 8 bits with a scale per row or per 128 columns, on
// gfx950: weights as they are loaded, activations that come from no norm.
//
// Memory bounds it: a row stays in the registers of its threads between its
// load, the reduction of its largest magnitude and the stores: 12,288 rows of
// 4096 bf16 columns take 30 us for 151 MB (5.0 TB/s), seven of 5003 4 us.
#include "norm_device.h"

namespace gdr {

namespace {

struct QuantArgs {
  const void* x;
  uint8_t* q;
  float* scale;
  int64_t x_stride;
  int rows, D, quant, group;
};

template <typename T, int NT, int VPT, bool PART>
__global__ __launch_bounds__(block_of<NT>()) void quantize_kernel(QuantArgs a) {
  __shared__ float lds[16];
  const int tid = NT == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int64_t row = NT == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (row >= a.rows) return;  // a whole wave; the barriers are for NT > 64 only
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride;
  float f[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    load8<T, PART>(x + column_of<PART>(i * NT + tid, a.D), a.D, f[i]);
  quantise_row<NT, VPT, PART>(f, row, tid, a.D, a.quant, a.group, a.q, a.scale, lds);
}

}  // namespace

gdr_status launch_quantize_rows(const gdr_quantize_problem* p, const void* x, void* q, float* scale,
                                hipStream_t st) {
  const QuantArgs a{x, reinterpret_cast<uint8_t*>(q), scale, p->x_stride, p->rows, p->D, p->quant,
                    p->group_size};
  const int nv = (p->D + 7) / 8;
  auto run = [&](auto t, auto nt, auto vpt, auto part) {
    using T = decltype(t);
    constexpr int NT = nt.value, VPT = vpt.value;
    GDR_LAUNCH("quantize_rows", (quantize_kernel<T, NT, VPT, part.value>),
               dim3((unsigned)(NT == 64 ? (p->rows + 3) / 4 : p->rows)), dim3(block_of<NT>()), st, a);
  };
  // the threads per row of the norms
  auto by_width = [&](auto t) {
    const std::false_type whole;
#define GDR_W(NT, VPT) \
  if (nv <= NT * VPT)  \
  return run(t, std::integral_constant<int, NT>(), std::integral_constant<int, VPT>(), whole)
    if (p->D < 8)
      return run(t, std::integral_constant<int, 64>(), std::integral_constant<int, 1>(),
                 std::true_type());
    GDR_W(64, 1);
    GDR_W(64, 2);
    GDR_W(256, 1);
    GDR_W(256, 2);
    GDR_W(256, 4);
    GDR_W(256, 8);
    GDR_W(1024, 4);
    GDR_W(1024, 8);
#undef GDR_W
  };
  if (p->dtype == GDR_BF16) by_width(__bf16());
  else if (p->dtype == GDR_FP16) by_width(_Float16());
  else by_width(float());
  return launch_status("quantize_rows");
}

}  // namespace gdr
