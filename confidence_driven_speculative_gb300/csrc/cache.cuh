// cache.cuh -- launch interfaces of the calls on drafted trees and on the
// caches of all layers (verify_tree.cu, commit_path.cu, update_pages.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dspark.h"

namespace dspark {

size_t tree_workspace_bytes();
cudaError_t launch_verify_tree(const dspark_tree &t, int sms, cudaStream_t s);

cudaError_t launch_commit_path(const dspark_cache &c, int B, int q_max, int max_pages, const int32_t *block_table,
                               const int32_t *seq_lens, const int32_t *path, int sms, cudaStream_t s);

size_t pages_workspace_bytes(int B, int num_pages);
cudaError_t launch_update_pages(const dspark_pages &p, int sms, cudaStream_t s);

}  // namespace dspark
