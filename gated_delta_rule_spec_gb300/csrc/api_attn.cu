// api_attn.cu -- the extern "C" entry points of the softmax-attention layers'
// step (declared and documented in include/gdn_spec.h): host-side checks, the rotary
// plan, kernel selection and stream-ordered launches.  Nothing here allocates,
// frees or synchronises, except gdn_spec_kv_read_status.
#include <cmath>
#include <cstdint>

#include "attn_common.cuh"
#include "launch_setup.cuh"

namespace gdnspec {

uint32_t data_wait_limit();

cudaError_t launch_kv_init(const KvArgs &C, cudaStream_t stream);
cudaError_t launch_kv_reserve(const KvArgs &C, const int32_t *slot_idx, int B, int T, const int32_t *n_tokens,
                              int32_t *done, cudaStream_t stream);
cudaError_t launch_kv_fork(const KvArgs &C, const int32_t *src_idx, const int32_t *dst_idx, int B, int32_t *done,
                           int es, cudaStream_t stream);
cudaError_t launch_kv_commit(const KvArgs &C, const int32_t *slot_idx, int B, int T, const int32_t *path,
                             const int32_t *accept_len, int es, cudaStream_t stream);
cudaError_t launch_kv_free(const KvArgs &C, const int32_t *slot_idx, int B, cudaStream_t stream);
int kv_alloc_max_rows();
int kv_move_max_window();
cudaError_t launch_rope(const gdn_spec_rope_plan *plan, int N, int heads, bool bf16, const int32_t *pos, const void *x,
                        int64_t x_stride, void *out, int64_t out_stride, bool transpose, cudaStream_t st);
cudaError_t launch_rope_append(const gdn_spec_rope_plan *plan, const KvArgs &C, bool bf16, int layer,
                               const int32_t *slot_idx, int B, int T, const int32_t *n_tokens, const int32_t *pos, int HQ,
                               const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                               int64_t v_stride, void *q_out, cudaStream_t st);
void tree_attn_cut(AttnArgs *A, int sms, int es);
cudaError_t launch_tree_attn(const AttnArgs &A, bool bf16, cudaStream_t st);
bool tree_attn_tc_supported(const KvArgs &C, int G, bool bf16);
void tree_attn_tc_cut(AttnArgs *A, int sms);
cudaError_t launch_tree_attn_tc(const AttnArgs &A, cudaStream_t st);

}  // namespace gdnspec

using namespace gdnspec;

namespace {

constexpr int kTreeMax = 64;            // drafted tokens of a window: bits of a mask
constexpr double kTwoPi = 6.283185307179586476925;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int cuda_rc(cudaError_t e) { return e == cudaSuccess ? GDN_SPEC_OK : GDN_SPEC_ECUDA; }
cudaStream_t as_stream(void *s) { return static_cast<cudaStream_t>(s); }
int elem_size(int io_dtype) { return io_dtype == GDN_SPEC_DTYPE_BF16 ? 2 : 4; }

int check_cache(const gdn_spec_kv_cache *c) {
    if (!c) return GDN_SPEC_EINVAL;
    if (c->io_dtype != GDN_SPEC_DTYPE_BF16 && c->io_dtype != GDN_SPEC_DTYPE_FP32) return GDN_SPEC_EDTYPE;
    if (c->n_layers <= 0 || c->num_pages <= 0 || c->HKV <= 0 || c->P <= 0 || c->D <= 0 || c->num_slots <= 0 ||
        c->max_pages <= 0)
        return GDN_SPEC_EINVAL;
    if (c->P & (c->P - 1)) return GDN_SPEC_EINVAL;
    if (c->D % 8 != 0) return GDN_SPEC_EALIGN;
    if (!c->k || !c->v || !c->page_table || !c->n_pages || !c->length || !c->ref || !c->free_bits || !c->status)
        return GDN_SPEC_EINVAL;
    if (!aligned16(c->k) || !aligned16(c->v)) return GDN_SPEC_EALIGN;
    if (c->P < 16 || c->P > 256 || c->D > 256) return GDN_SPEC_EUNSUPPORTED;
    // token rows of the pool, and of a slot, are held in 31 bits
    if ((int64_t)c->num_pages * c->P > INT32_MAX || (int64_t)c->max_pages * c->P > INT32_MAX) return GDN_SPEC_EUNSUPPORTED;
    if ((int64_t)c->n_layers * c->HKV > (1 << 20)) return GDN_SPEC_EUNSUPPORTED;
    return GDN_SPEC_OK;
}

KvArgs kv_args(const gdn_spec_kv_cache *c) {
    KvArgs C;
    C.n_layers = c->n_layers;
    C.num_pages = c->num_pages;
    C.HKV = c->HKV;
    C.P = c->P;
    C.logP = __builtin_ctz((unsigned)c->P);
    C.D = c->D;
    C.num_slots = c->num_slots;
    C.max_pages = c->max_pages;
    C.k = c->k;
    C.v = c->v;
    C.page_table = c->page_table;
    C.n_pages = c->n_pages;
    C.length = c->length;
    C.ref = c->ref;
    C.free_bits = c->free_bits;
    C.status = c->status;
    return C;
}

int check_plan(const gdn_spec_rope_plan *p) {
    if (!p) return GDN_SPEC_EINVAL;
    if (p->D <= 0 || p->rot < 2 || p->rot > p->D || p->rot % 2) return GDN_SPEC_EINVAL;
    if (p->layout != GDN_SPEC_ROPE_HALF && p->layout != GDN_SPEC_ROPE_INTERLEAVED) return GDN_SPEC_EINVAL;
    if (p->D % 8 != 0) return GDN_SPEC_EALIGN;
    if (p->D > 256) return GDN_SPEC_EUNSUPPORTED;
    return GDN_SPEC_OK;
}

// Radians per position as a fraction of 2^64 of a turn (whole turns fall away).
uint64_t turn_bits(double f) {
    double t = f / kTwoPi;
    t -= std::floor(t);
    // in two halves, so that the product stays inside the double's range of whole numbers
    const double hi = std::floor(t * 4294967296.0);
    const double lo = std::floor((t * 4294967296.0 - hi) * 4294967296.0 + 0.5);
    return (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(lo);
}

// Block of checks of one attention call that do not need a device.
int check_attn(const gdn_spec_kv_cache *c, int32_t B, int32_t T, int32_t HQ) {
    const int rc = check_cache(c);
    if (rc) return rc;
    if (B < 0 || T <= 0 || HQ <= 0 || HQ % c->HKV != 0) return GDN_SPEC_EINVAL;
    if (T > kTreeMax || HQ / c->HKV > 4096) return GDN_SPEC_EUNSUPPORTED;
    // the line of key/value tiles (of 32 tokens, a row's last one begun, and gaps of at most 8) and the tokens are
    // counted in 31 bits
    if ((double)B * (((int64_t)c->max_pages * c->P + 31) / 32 + 8) * c->HKV > 2.0e9) return GDN_SPEC_EUNSUPPORTED;
    if ((int64_t)B * T > INT32_MAX) return GDN_SPEC_EUNSUPPORTED;
    return GDN_SPEC_OK;
}

int device_sms(int *sms) {
    static KernelSetup none;   // the SM count alone
    const cudaError_t e = kernel_setup(none, nullptr, 0, sms);
    return cuda_rc(e);
}

bool attn_on_tc(const gdn_spec_kv_cache *c, int32_t HQ) {
    return tree_attn_tc_supported(kv_args(c), HQ / c->HKV, c->io_dtype == GDN_SPEC_DTYPE_BF16);
}

int attn_args(const gdn_spec_kv_cache *c, int32_t B, int32_t T, int32_t HQ, AttnArgs *A) {
    A->C = kv_args(c);
    A->layer = 0;
    A->B = B;
    A->T = T;
    A->HQ = HQ;
    A->G = HQ / c->HKV;
    int sms;
    const int rc = device_sms(&sms);
    if (rc) return rc;
    if (attn_on_tc(c, HQ)) tree_attn_tc_cut(A, sms); else tree_attn_cut(A, sms, elem_size(c->io_dtype));
    return GDN_SPEC_OK;
}

// Workspace: pieces' sums, their maxima and sums (one group cuts nothing), the chunks' notes.
int64_t part_rows(const AttnArgs &A) { return A.groups < 2 ? 0 : (int64_t)A.groups * A.NQT * 2 * A.MT; }
int64_t workspace_bytes_of(const AttnArgs &A) {
    return part_rows(A) * ((int64_t)A.C.D * 4 + 8) + (int64_t)A.groups * sizeof(AttnCut);
}

}  // namespace

extern "C" {

int gdn_spec_kv_init(const gdn_spec_kv_cache *cache, void *stream) {
    const int rc = check_cache(cache);
    if (rc) return rc;
    return cuda_rc(launch_kv_init(kv_args(cache), as_stream(stream)));
}

int gdn_spec_kv_reserve(const gdn_spec_kv_cache *cache, const int32_t *slot_idx, int32_t B, int32_t T,
                        const int32_t *n_tokens, int32_t *done, void *stream) {
    const int rc = check_cache(cache);
    if (rc) return rc;
    if (B < 0 || T < 0) return GDN_SPEC_EINVAL;
    if (B == 0) return GDN_SPEC_OK;
    if (!slot_idx || !done) return GDN_SPEC_EINVAL;
    if (B > kv_alloc_max_rows() || (int64_t)B * cache->max_pages > INT32_MAX) return GDN_SPEC_EUNSUPPORTED;
    return cuda_rc(launch_kv_reserve(kv_args(cache), slot_idx, B, T, n_tokens, done, as_stream(stream)));
}

int gdn_spec_kv_fork(const gdn_spec_kv_cache *cache, const int32_t *src_idx, const int32_t *dst_idx, int32_t B,
                     int32_t *done, void *stream) {
    const int rc = check_cache(cache);
    if (rc) return rc;
    if (B < 0) return GDN_SPEC_EINVAL;
    if (B == 0) return GDN_SPEC_OK;
    if (!src_idx || !dst_idx || !done) return GDN_SPEC_EINVAL;
    if (B > kv_alloc_max_rows()) return GDN_SPEC_EUNSUPPORTED;
    return cuda_rc(launch_kv_fork(kv_args(cache), src_idx, dst_idx, B, done, elem_size(cache->io_dtype),
                                  as_stream(stream)));
}

int gdn_spec_kv_commit(const gdn_spec_kv_cache *cache, const int32_t *slot_idx, int32_t B, int32_t T,
                       const int32_t *path, const int32_t *accept_len, void *stream) {
    const int rc = check_cache(cache);
    if (rc) return rc;
    if (B < 0 || T <= 0) return GDN_SPEC_EINVAL;
    if (B == 0) return GDN_SPEC_OK;
    if (!slot_idx || !accept_len) return GDN_SPEC_EINVAL;
    if (path && T > kv_move_max_window()) return GDN_SPEC_EUNSUPPORTED;
    return cuda_rc(launch_kv_commit(kv_args(cache), slot_idx, B, T, path, accept_len, elem_size(cache->io_dtype),
                                    as_stream(stream)));
}

int gdn_spec_kv_free(const gdn_spec_kv_cache *cache, const int32_t *slot_idx, int32_t B, void *stream) {
    const int rc = check_cache(cache);
    if (rc) return rc;
    if (B < 0) return GDN_SPEC_EINVAL;
    if (B == 0) return GDN_SPEC_OK;
    if (!slot_idx) return GDN_SPEC_EINVAL;
    return cuda_rc(launch_kv_free(kv_args(cache), slot_idx, B, as_stream(stream)));
}

int gdn_spec_kv_read_status(const gdn_spec_kv_cache *cache, uint32_t *host_out, int32_t clear, void *stream) {
    const int rc = check_cache(cache);
    if (rc) return rc;
    if (!host_out) return GDN_SPEC_EINVAL;
    const cudaStream_t st = as_stream(stream);
    cudaError_t e = cudaMemcpyAsync(host_out, cache->status, sizeof(uint32_t), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess && clear) e = cudaMemsetAsync(cache->status, 0, sizeof(uint32_t), st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    return cuda_rc(e);
}

int gdn_spec_rope_init_freqs(gdn_spec_rope_plan *plan, int32_t D, int32_t rot, int32_t layout, const double *freqs,
                             double mscale) {
    if (!plan || !freqs) return GDN_SPEC_EINVAL;
    gdn_spec_rope_plan p = {};
    p.D = D;
    p.rot = rot;
    p.layout = layout;
    p.mscale = (float)mscale;
    const int rc = check_plan(&p);
    if (rc) return rc;
    if (!std::isfinite(p.mscale)) return GDN_SPEC_EINVAL;   // as the fp32 number that is kept
    for (int i = 0; i < rot / 2; ++i) {
        if (!std::isfinite(freqs[i])) return GDN_SPEC_EINVAL;
        p.freq[i] = turn_bits(freqs[i]);
    }
    *plan = p;
    return GDN_SPEC_OK;
}

int gdn_spec_rope_init(gdn_spec_rope_plan *plan, int32_t D, int32_t rot, int32_t layout, double base,
                       const gdn_spec_rope_scaling *scaling) {
    if (!plan || rot < 2 || rot > 256 || !(base > 1.0) || !std::isfinite(base)) return GDN_SPEC_EINVAL;
    const int kind = scaling ? scaling->kind : GDN_SPEC_ROPE_NONE;
    if (kind < GDN_SPEC_ROPE_NONE || kind > GDN_SPEC_ROPE_BANDS) return GDN_SPEC_EINVAL;
    const double factor = kind == GDN_SPEC_ROPE_NONE ? 1.0 : scaling->factor;
    if (!(factor >= 1.0) || !std::isfinite(factor)) return GDN_SPEC_EINVAL;
    if (kind == GDN_SPEC_ROPE_NTK) {
        if (rot <= 2) return GDN_SPEC_EINVAL;
        base *= std::pow(factor, rot / (rot - 2.0));
    }
    double f[128], mscale = 1.0;
    const int pairs = rot / 2;
    for (int i = 0; i < pairs; ++i) f[i] = std::pow(base, -2.0 * i / rot);
    if (kind == GDN_SPEC_ROPE_LINEAR) {
        for (int i = 0; i < pairs; ++i) f[i] /= factor;
    } else if (kind == GDN_SPEC_ROPE_YARN) {
        if (!(scaling->original > 0.0) || !(scaling->low > scaling->high) || !(scaling->high > 0.0)) return GDN_SPEC_EINVAL;
        // the pair (as a real number) that turns n times in `original` positions
        const auto pair_of = [&](double n) { return rot * std::log(scaling->original / (n * kTwoPi)) / (2.0 * std::log(base)); };
        const double first = std::fmax(std::floor(pair_of(scaling->low)), 0.0);
        const double last = std::fmin(std::ceil(pair_of(scaling->high)), rot - 1.0);
        const double span = std::fmax(last - first, 1e-3);
        for (int i = 0; i < pairs; ++i) {
            const double ramp = std::fmin(std::fmax((i - first) / span, 0.0), 1.0);
            f[i] = f[i] / factor * ramp + f[i] * (1.0 - ramp);
        }
        mscale = 0.1 * std::log(factor) + 1.0;
    } else if (kind == GDN_SPEC_ROPE_BANDS) {
        if (!(scaling->original > 0.0) || !(scaling->high > scaling->low)) return GDN_SPEC_EINVAL;
        for (int i = 0; i < pairs; ++i) {
            const double turns = scaling->original * f[i] / kTwoPi;
            const double mix = std::fmin(std::fmax((turns - scaling->low) / (scaling->high - scaling->low), 0.0), 1.0);
            f[i] = (1.0 - mix) * f[i] / factor + mix * f[i];
        }
    }
    return gdn_spec_rope_init_freqs(plan, D, rot, layout, f, mscale);
}

int gdn_spec_rope(const gdn_spec_rope_plan *plan, int32_t N, int32_t heads, int32_t io_dtype, const int32_t *pos,
                  const void *x, int64_t x_stride, void *out, int64_t out_stride, int32_t transpose, void *stream) {
    const int rc = check_plan(plan);
    if (rc) return rc;
    if (io_dtype != GDN_SPEC_DTYPE_BF16 && io_dtype != GDN_SPEC_DTYPE_FP32) return GDN_SPEC_EDTYPE;
    if (N < 0 || heads <= 0) return GDN_SPEC_EINVAL;
    const int64_t row = (int64_t)heads * plan->D;
    if (x_stride < row || out_stride < row || (x && x == out && x_stride != out_stride)) return GDN_SPEC_EINVAL;
    if (x_stride % 8 != 0 || out_stride % 8 != 0) return GDN_SPEC_EALIGN;
    if (row > (1 << 22)) return GDN_SPEC_EUNSUPPORTED;
    if (N == 0) return GDN_SPEC_OK;
    if (!pos || !x || !out) return GDN_SPEC_EINVAL;
    if (!aligned16(x) || !aligned16(out)) return GDN_SPEC_EALIGN;
    return cuda_rc(launch_rope(plan, N, heads, io_dtype == GDN_SPEC_DTYPE_BF16, pos, x, x_stride, out, out_stride,
                               transpose != 0, as_stream(stream)));
}

int gdn_spec_rope_append(const gdn_spec_rope_plan *plan, const gdn_spec_kv_cache *cache, int32_t layer,
                         const int32_t *slot_idx, int32_t B, int32_t T, const int32_t *n_tokens, const int32_t *pos,
                         int32_t HQ, const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                         int64_t v_stride, void *q_out, void *stream) {
    int rc = check_plan(plan);
    if (rc) return rc;
    if ((rc = check_cache(cache))) return rc;
    if (plan->D != cache->D) return GDN_SPEC_EINVAL;
    if (layer < 0 || layer >= cache->n_layers || B < 0 || T <= 0 || HQ <= 0) return GDN_SPEC_EINVAL;
    const int64_t kv_row = (int64_t)cache->HKV * cache->D, q_row = (int64_t)HQ * cache->D;
    if (q_stride < q_row || k_stride < kv_row || v_stride < kv_row) return GDN_SPEC_EINVAL;
    if (q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0) return GDN_SPEC_EALIGN;
    if (q_row + 2 * kv_row > (1 << 22) || (int64_t)B * T > INT32_MAX) return GDN_SPEC_EUNSUPPORTED;
    if (B == 0) return GDN_SPEC_OK;
    if (!slot_idx || !q || !k || !v || !q_out) return GDN_SPEC_EINVAL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out)) return GDN_SPEC_EALIGN;
    return cuda_rc(launch_rope_append(plan, kv_args(cache), cache->io_dtype == GDN_SPEC_DTYPE_BF16, layer, slot_idx, B, T,
                                      n_tokens, pos, HQ, q, q_stride, k, k_stride, v, v_stride, q_out,
                                      as_stream(stream)));
}

const char *gdn_spec_tree_attn_path(const gdn_spec_kv_cache *cache, int32_t T, int32_t HQ) {
    if (check_attn(cache, 0, T, HQ) != GDN_SPEC_OK) return nullptr;
    return attn_on_tc(cache, HQ) ? "tc" : "generic";
}

int64_t gdn_spec_tree_attn_workspace(const gdn_spec_kv_cache *cache, int32_t B, int32_t T, int32_t HQ) {
    int rc = check_attn(cache, B, T, HQ);
    if (rc) return rc;
    AttnArgs A = {};
    if ((rc = attn_args(cache, B, T, HQ, &A))) return rc;
    return workspace_bytes_of(A);
}

int gdn_spec_tree_attn(const gdn_spec_kv_cache *cache, int32_t layer, const int32_t *slot_idx, int32_t B, int32_t T,
                       int32_t HQ, const void *q, const uint64_t *tree_mask, const int32_t *tree_len, float scale,
                       void *out, float *lse, void *workspace, int64_t workspace_bytes, void *stream) {
    int rc = check_attn(cache, B, T, HQ);
    if (rc) return rc;
    // scores are scaled in powers of two, by a factor that has to be finite too
    const float scale_log2 = (float)((double)scale * 1.4426950408889634);
    if (layer < 0 || layer >= cache->n_layers || !(scale > 0.0f) || !std::isfinite(scale_log2)) return GDN_SPEC_EINVAL;
    if (B == 0) return GDN_SPEC_OK;
    if (!slot_idx || !q || !out || !workspace) return GDN_SPEC_EINVAL;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return GDN_SPEC_EALIGN;
    AttnArgs A = {};
    if ((rc = attn_args(cache, B, T, HQ, &A))) return rc;
    const int64_t rows = part_rows(A);
    if (workspace_bytes < workspace_bytes_of(A)) return GDN_SPEC_EINVAL;
    A.layer = layer;
    A.slot_idx = slot_idx;
    A.tree_mask = tree_mask;
    A.tree_len = tree_len;
    A.scale_log2 = scale_log2;
    A.q = q;
    A.out = out;
    A.lse = lse;
    A.part_o = static_cast<float4 *>(workspace);
    A.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + rows * cache->D * 4);
    A.cuts = reinterpret_cast<AttnCut *>(static_cast<char *>(workspace) + rows * ((int64_t)cache->D * 4 + 8));
    A.wait_limit = data_wait_limit();
    if (attn_on_tc(cache, HQ)) return cuda_rc(launch_tree_attn_tc(A, as_stream(stream)));
    return cuda_rc(launch_tree_attn(A, cache->io_dtype == GDN_SPEC_DTYPE_BF16, as_stream(stream)));
}

}  // extern "C"
