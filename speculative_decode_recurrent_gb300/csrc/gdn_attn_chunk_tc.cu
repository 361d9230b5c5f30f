#include "chunk_common.h"
namespace gdn {
int64_t chunk_tc_workspace(const gdn_page_cache *, const gdn_attn_dims *) { return 0; }
int chunk_tc(const gdn_page_cache *, const gdn_attn_dims *, ChunkArgs, cudaStream_t) { return GDN_ERR_DIMS; }
}
