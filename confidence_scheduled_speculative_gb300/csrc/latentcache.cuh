// latentcache.cuh -- the paged latent cache as the kernels see it: one head of
// latent_dim + rope_dim elements a token, which kvcache.cuh's addressing serves.
#pragma once

#include "kvcache.cuh"

namespace dspark {

// Host-side checks of a latent cache; DSPARK_OK or the call's error.
inline int latent_check(const dspark_latent_cache *c) {
    if (!c || !c->data || !c->block_table) return DSPARK_ERR_INVALID_ARG;
    if (c->dtype != DSPARK_DTYPE_BF16 && c->dtype != DSPARK_DTYPE_F32) return DSPARK_ERR_INVALID_ARG;
    if (c->n_pages < 1 || c->page_size < 1 || c->n_requests < 1 || c->table_width < 1 ||
        c->page_stride < 0 || c->token_stride < 0)
        return DSPARK_ERR_INVALID_ARG;
    if (c->latent_dim < 2 || c->latent_dim > DSPARK_MAX_LATENT_DIM || c->latent_dim % 2 ||
        c->rope_dim < 2 || c->rope_dim > DSPARK_MAX_LATENT_ROPE || c->rope_dim % 2)
        return DSPARK_ERR_UNSUPPORTED;
    return DSPARK_OK;
}

inline KvView latent_view(const dspark_latent_cache &c) {
    KvView w = {};
    w.k = w.v = static_cast<unsigned char *>(c.data);
    w.table = c.block_table;
    w.page_stride = c.page_stride;
    w.token_stride = c.token_stride;
    w.n_pages = c.n_pages;
    w.page_size = c.page_size;
    w.n_kv_heads = 1;
    w.head_dim = c.latent_dim + c.rope_dim;
    w.n_requests = c.n_requests;
    w.table_width = c.table_width;
    return w;
}

}  // namespace dspark
