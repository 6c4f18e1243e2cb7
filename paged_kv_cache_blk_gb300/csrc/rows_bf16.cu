// The kernels of rows.cuh for bf16 pools.
#include "rows.cuh"

namespace pkv {

cudaError_t launch_rows_bf16(const RowsParams& p, int D, bool tree, long long grid, int dev,
                             cudaStream_t s) {
  return D == 64 ? launch_rows_d<PKV_BF16, 64>(p, tree, grid, dev, s)
                 : launch_rows_d<PKV_BF16, 128>(p, tree, grid, dev, s);
}

int rows_ctas_bf16(int D, int unit_rows) {
  return D == 64 ? rows_ctas_d<PKV_BF16, 64>(unit_rows) : rows_ctas_d<PKV_BF16, 128>(unit_rows);
}

}  // namespace pkv
