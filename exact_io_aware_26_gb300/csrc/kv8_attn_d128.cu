// kv8_attn_d128.cu -- the 8-bit cache attention's kernels for head size 128 (kv_attn.cuh).
#include "kv_attn.cuh"

namespace fa {
template cudaError_t launch_kv_attention<Kv8Block<128>>(const Kv4AttnArgs&, bool, int, int, int, cudaStream_t);
template int kv_clusters_at_once<Kv8Block<128>>(int, int);
}
