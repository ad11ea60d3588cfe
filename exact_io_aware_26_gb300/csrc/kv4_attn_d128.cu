// kv4_attn_d128.cu -- the cache attention's kernels for head size 128 (kv4_attn.cuh).
#include "kv4_attn.cuh"

namespace fa {
template cudaError_t launch_kv4_attention_d<128>(const Kv4AttnArgs&, bool, int, int, int, cudaStream_t);
template int kv4_clusters_at_once<128>(int, int);
}
