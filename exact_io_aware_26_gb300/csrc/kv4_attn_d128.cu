// kv4_attn_d128.cu -- the 4-bit cache attention's kernels for head size 128 (kv_attn.cuh).
#include "kv_attn.cuh"

namespace fa {
template cudaError_t launch_kv_attention<KvBlock<128>>(const Kv4AttnArgs&, bool, int, int, int, cudaStream_t);
template int kv_clusters_at_once<KvBlock<128>>(int, int);
}
