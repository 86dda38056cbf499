/*
 * gdn_spec_attn_example.c -- one speculative step of a softmax-attention layer through
 * the C ABI of libgdnspec (include/gdn_spec.h): rotary positions and append, attention of
 * the drafted tree, then, once for all layers, the commit of the accepted path and
 * the pages of the next window.
 *
 * Every pointer in the cache and the arguments is caller-owned device memory of the
 * current CUDA device; no call allocates, and the calls are ordered on `stream`, so
 * the step can be captured in a CUDA graph.  Host-only example: compiles against the
 * header alone (link libgdnspec.so to run it).
 */
#include <stdint.h>
#include <stdio.h>

#include "gdn_spec.h"

int gdn_spec_attn_example_step(const gdn_spec_kv_cache *cache, const int32_t *slot_idx, int32_t B,
                               const void *qkv, const int32_t *pos, const uint64_t *tree_mask,
                               const int32_t *path, const int32_t *accept_len, void *q_rot,
                               void *out, void *workspace, int64_t workspace_bytes, int32_t *done,
                               void *stream)
{
    /* a window of 8 drafted nodes, 16 query heads; the first 64 dims of a head are rotated */
    const int32_t T = 8, HQ = 16;
    gdn_spec_rope_plan plan;
    int rc = gdn_spec_rope_init(&plan, cache->D, 64, GDN_SPEC_ROPE_HALF, 1.0e6, NULL);

    /* q, k and v are slices of one projection's output [B, T, HQ + 2 HKV, D] (bf16 here) */
    const int64_t stride = (int64_t)(HQ + 2 * cache->HKV) * cache->D;
    const char *q = (const char *)qkv;
    const char *k = q + 2 * (int64_t)HQ * cache->D;
    const char *v = k + 2 * (int64_t)cache->HKV * cache->D;
    for (int32_t layer = 0; !rc && layer < cache->n_layers; ++layer) {
        rc = gdn_spec_rope_append(&plan, cache, layer, slot_idx, B, T, NULL, pos, HQ, q, stride, k,
                                  stride, v, stride, q_rot, stream);
        if (!rc)
            rc = gdn_spec_tree_attn(cache, layer, slot_idx, B, T, HQ, q_rot, tree_mask, NULL,
                                    0.0625f, out, NULL, workspace, workspace_bytes, stream);
    }
    /* path and accept_len are produced on the device by the sampler */
    if (!rc) rc = gdn_spec_kv_commit(cache, slot_idx, B, T, path, accept_len, stream);
    if (!rc) rc = gdn_spec_kv_reserve(cache, slot_idx, B, T, NULL, done, stream);
    if (rc) {
        fprintf(stderr, "%s\n", gdn_spec_strerror(rc));
        return rc;
    }
    uint32_t st = 0;
    rc = gdn_spec_kv_read_status(cache, &st, /*clear=*/1, stream);
    if (!rc && st) fprintf(stderr, "device status 0x%x\n", st);
    return rc;
}
