// The kernels of rows.cuh for fp32 pools.
#include "rows.cuh"

namespace pkv {

cudaError_t launch_rows_f32(const RowsParams& p, int D, bool tree, long long grid, int dev,
                            cudaStream_t s) {
  return D == 64 ? launch_rows_d<PKV_F32, 64>(p, tree, grid, dev, s)
                 : launch_rows_d<PKV_F32, 128>(p, tree, grid, dev, s);
}

int rows_ctas_f32(int D, int unit_rows) {
  return D == 64 ? rows_ctas_d<PKV_F32, 64>(unit_rows) : rows_ctas_d<PKV_F32, 128>(unit_rows);
}

}  // namespace pkv
