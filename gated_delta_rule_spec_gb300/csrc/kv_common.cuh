// kv_common.cuh -- the paged key/value cache of the softmax-attention layers as
// the kernels see it, and the checks of one batch row that every call makes
// before it touches a page.
#pragma once

#include "common.cuh"

namespace gdnspec {

struct KvArgs {
    int n_layers, num_pages, HKV, P, logP, D, num_slots, max_pages;
    void *k, *v;
    int32_t *page_table, *n_pages, *length, *ref;
    uint32_t *free_bits, *status;
};

// Committed length of `slot`, or -1 with *bits set when the slot or its counts
// are out of range (*bits = 0: a padding row).
__device__ __forceinline__ int kv_slot_length(const KvArgs &C, int slot, int *n_pages, uint32_t *bits) {
    *bits = 0;
    *n_pages = 0;
    if (slot < 0) return -1;
    if (slot >= C.num_slots) { *bits = GDN_SPEC_ST_SLOT_OOR; return -1; }
    const int len = C.length[slot], np = C.n_pages[slot];
    if (len < 0 || np < 0 || np > C.max_pages || (int64_t)len > (int64_t)np * C.P) {
        *bits = GDN_SPEC_ST_CURSOR_CORRUPT;
        return -1;
    }
    *n_pages = np;
    return len;
}

// The row of `slot` with `cnt` tokens behind its committed ones (cnt_max: the
// window): its committed length, or -1 with *bits set when it is not computed.
__device__ __forceinline__ int kv_row(const KvArgs &C, int slot, int cnt, int cnt_max, uint32_t *bits) {
    int np;
    const int len = kv_slot_length(C, slot, &np, bits);
    if (len < 0) return -1;
    if (cnt < 0 || cnt > cnt_max) { *bits = GDN_SPEC_ST_ACCEPT_RANGE; return -1; }
    if ((int64_t)len + cnt > (int64_t)np * C.P) { *bits = GDN_SPEC_ST_NO_PAGES; return -1; }
    return len;
}

// Row of the pool's [num_pages * P] token rows that holds token `tok` of `slot`,
// or -1 when the table's entry is not a page.
__device__ __forceinline__ int64_t kv_token_row(const KvArgs &C, int slot, int tok) {
    const int page = C.page_table[(int64_t)slot * C.max_pages + (tok >> C.logP)];
    if (page < 0 || page >= C.num_pages) return -1;
    return ((int64_t)page << C.logP) + (tok & (C.P - 1));
}

// Element offset of head h of a token row in layer `layer`.
__device__ __forceinline__ int64_t kv_elem(const KvArgs &C, int layer, int h, int64_t row) {
    const int64_t page = row >> C.logP;
    return ((((int64_t)layer * C.num_pages + page) * C.HKV + h) * C.P + (row & (C.P - 1))) * C.D;
}

}  // namespace gdnspec
