// The kernels that choose a row's pages and attend to them at once, in a
// translation unit of their own (they take as long to compile as all others).
#include "pa_sparse_attend.cuh"

namespace pa {
namespace sparse {

pa_status launch_chosen(int head_dim, int block_size, bool fp8, const CUtensorMap &tk, const CUtensorMap &tv, const Args &a,
                        int num_rows, int splits, int warps, cudaStream_t stream) {
    return launch_any<kChoose>(head_dim, block_size, fp8, tk, tv, a, num_rows, splits, warps, stream, a.group);
}

}  // namespace sparse
}  // namespace pa
