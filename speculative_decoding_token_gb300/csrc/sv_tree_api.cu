// sv_tree_api.cu -- the C ABI of the token-tree calls (declared in
// include/specverify.h): handle, host-side argument checks, launches.
#include <cmath>
#include <algorithm>
#include <new>

#include "sv_host.h"
#include "sv_tree.h"

struct specverify_tree_ctx {
    int device = 0;
    int num_sms = 0;
    int32_t max_batch = 0;
    int64_t max_moves = 0;
    uint64_t wait_ns = sv::kDefaultWaitNs;
    void *ws = nullptr;
    size_t ws_bytes = 0;
    int32_t *status = nullptr;
    int32_t *move_src = nullptr, *move_dst = nullptr, *move_cnt = nullptr;
    void *attn = nullptr;
};

namespace {

using sv::DeviceGuard;
using sv::map_cuda;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether [a, a + n) and [b, b + m) share a byte.
bool overlap(const void *a, int64_t n, const void *b, int64_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)m && y < x + (uintptr_t)n;
}

// A strided layout in bytes, to see whether its elements, or those of two buffers
// laid out alike, keep to memory of their own: sorted by size, each stride has to be
// at least the extent of what lies below it. Every view that slicing and transposing
// make of a plain buffer is such a one.
struct Layout {
    struct Dim {
        int64_t count, stride;
    } dim[6];
    int dims = 0;
    int64_t inner;  // contiguous bytes of an element

    explicit Layout(int64_t bytes) : inner(bytes) {}
    Layout &add(int64_t count, int64_t stride) {
        if (count > 1) dim[dims++] = {count, stride};
        return *this;
    }
    bool apart() const {
        Dim d[6];
        std::copy(dim, dim + dims, d);
        std::sort(d, d + dims, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
        __int128 span = inner;
        for (int i = 0; i < dims; ++i) {
            if (d[i].stride < span) return false;
            span += (__int128)d[i].stride * (d[i].count - 1);
        }
        return true;
    }
    // of a buffer at a and another at b, both of this layout
    bool apart(const void *a, const void *b) const {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
        return Layout(*this).add(2, (int64_t)(x < y ? y - x : x - y)).apart();
    }
};

Layout rows_layout(int64_t rows, int64_t heads, int64_t d, int64_t rs, int64_t hs) {
    return Layout(d * 2).add(rows, rs * 2).add(heads, hs * 2);
}

Layout kv_layout(const specverify_cache *c) {
    return Layout(c->head_dim * 2)
        .add(c->layers, c->layer_stride * 2)
        .add(c->num_pages, c->page_stride * 2)
        .add(c->kv_heads, c->head_stride * 2)
        .add(c->page_size, c->token_stride * 2);
}

Layout mass_layout(const specverify_cache *c) {
    return Layout(4)
        .add(c->layers, c->mass_layer_stride * 4)
        .add(c->num_pages, c->mass_page_stride * 4)
        .add(c->kv_heads, c->mass_head_stride * 4)
        .add(c->page_size, c->mass_token_stride * 4);
}

// Whether a call may write the cache's keys, values, masses and positions.
bool writable(const specverify_cache *c) {
    if (!kv_layout(c).apart(c->k, c->v)) return false;
    const Layout m = mass_layout(c);
    if (c->mass && c->pos) return m.apart(c->mass, c->pos);
    return (!c->mass && !c->pos) || m.apart();
}

int check_cache(const specverify_cache *c, int32_t B, bool one_layer) {
    if (!c) return SPECVERIFY_ERR_INVALID_ARG;
    if (c->dtype != SPECVERIFY_BF16 && c->dtype != SPECVERIFY_FP16)
        return SPECVERIFY_ERR_INVALID_ARG;
    if (c->layers < 1 || (one_layer && c->layers != 1)) return SPECVERIFY_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->num_pages > INT32_MAX || c->page_size < 8 ||
        c->page_size % 8 != 0 || c->kv_heads < 1 || (c->head_dim != 64 && c->head_dim != 128))
        return SPECVERIFY_ERR_INVALID_ARG;
    if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return SPECVERIFY_ERR_INVALID_ARG;
    // 8 elements are 16 bytes; a tensor map's strides end below 2^40 bytes
    const int64_t most = (int64_t)1 << 38;
    for (const int64_t s : {c->layer_stride, c->page_stride, c->head_stride, c->token_stride})
        if (s < 0 || s % 8 != 0 || s > most) return SPECVERIFY_ERR_INVALID_ARG;
    if ((c->layers > 1 && c->layer_stride == 0) || (c->num_pages > 1 && c->page_stride == 0) ||
        (c->kv_heads > 1 && c->head_stride == 0) || c->token_stride == 0)
        return SPECVERIFY_ERR_INVALID_ARG;
    if (c->max_pages < 1 || c->table_stride < c->max_pages || (B > 0 && !c->page_table) ||
        (int64_t)c->max_pages * c->page_size > ((int64_t)1 << 30))
        return SPECVERIFY_ERR_INVALID_ARG;
    if ((int64_t)B * c->kv_heads > INT32_MAX) return SPECVERIFY_ERR_INVALID_ARG;
    return SPECVERIFY_OK;
}

int check_tree(const specverify_tree_ctx *h, const specverify_tree *t, bool tokens) {
    if (!h || !t) return SPECVERIFY_ERR_INVALID_ARG;
    if (t->B < 0 || t->B > h->max_batch) return SPECVERIFY_ERR_INVALID_ARG;
    if (t->max_nodes < 1 || t->max_nodes > sv::kMaxNodes) return SPECVERIFY_ERR_INVALID_ARG;
    if (t->B == 0) return SPECVERIFY_OK;
    if (!t->row_off || !t->nodes || !t->parent || (tokens && !t->tokens))
        return SPECVERIFY_ERR_INVALID_ARG;
    return SPECVERIFY_OK;
}

// Rows of [rows, heads, d] with their strides.
int check_rows(const specverify_cache *c, const void *p, int64_t rows, int32_t heads, int64_t rs,
               int64_t hs) {
    if (rows < 0 || rows > INT32_MAX || heads < 1 || heads % c->kv_heads != 0)
        return SPECVERIFY_ERR_INVALID_ARG;
    if (rows > 0 && (!p || !aligned16(p))) return SPECVERIFY_ERR_INVALID_ARG;
    if (rs < 0 || hs < 0 || rs % 8 != 0 || hs % 8 != 0) return SPECVERIFY_ERR_INVALID_ARG;
    return SPECVERIFY_OK;
}

sv::CacheParams cache_params(const specverify_cache *c) {
    sv::CacheParams p{};
    p.k = static_cast<char *>(c->k);
    p.v = static_cast<char *>(c->v);
    p.ls = c->layer_stride * 2;
    p.ps = c->page_stride * 2;
    p.hs = c->head_stride * 2;
    p.ts = c->token_stride * 2;
    p.mass = c->mass;
    p.pos = c->pos;
    p.mls = c->mass_layer_stride;
    p.mps = c->mass_page_stride;
    p.mhs = c->mass_head_stride;
    p.mts = c->mass_token_stride;
    p.table = c->page_table;
    p.table_stride = c->table_stride;
    p.num_pages = c->num_pages;
    p.max_pages = c->max_pages;
    sv::set_page(p, c->page_size);
    p.kv_heads = c->kv_heads;
    p.d = c->head_dim;
    p.layers = c->layers;
    p.fp16 = c->dtype == SPECVERIFY_FP16;
    return p;
}

sv::TreeParams tree_params(const specverify_tree *t) {
    return {t->row_off, t->nodes, t->parent, t->tokens, t->B, t->max_nodes};
}

bool good_scale(float scale) { return scale > 0.0f && std::isfinite(scale * 1.44269504f); }

}  // namespace

extern "C" {

int specverify_tree_create(specverify_tree_t *out, int device, int32_t max_batch,
                           int64_t max_moves) {
    if (!out) return SPECVERIFY_ERR_INVALID_ARG;
    *out = nullptr;
    if (max_batch < 1 || max_batch > 65535 || max_moves < 0 || max_moves > ((int64_t)1 << 36) ||
        device < 0)
        return SPECVERIFY_ERR_INVALID_ARG;
    const int found = sv::check_device(device);
    if (found != SPECVERIFY_OK) return found;
    DeviceGuard guard(device);
    if (guard.err != cudaSuccess) return map_cuda(guard.err);
    specverify_tree_ctx *h = new (std::nothrow) specverify_tree_ctx();
    if (!h) return SPECVERIFY_ERR_OOM;
    h->device = device;
    h->max_batch = max_batch;
    h->max_moves = max_moves;
    cudaError_t e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, device);
    if (e == cudaSuccess) e = sv::prepare_tree();
    if (e == cudaSuccess) e = sv::prepare_accumulate();
    if (e == cudaSuccess) e = sv::prepare_evict();
    // an item moves at least one token, so max_moves bounds the items as well
    const size_t lists = sizeof(int32_t) * (size_t)max_moves;
    h->ws_bytes = 256 + 3 * ((lists + 255) / 256 * 256) + sv::attn_workspace(h->num_sms);
    if (e == cudaSuccess) e = cudaMalloc(&h->ws, h->ws_bytes);
    if (e == cudaSuccess) e = cudaMemset(h->ws, 0, 256);
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);  // the caller's streams need not wait for it
    if (e != cudaSuccess) {
        if (h->ws) cudaFree(h->ws);
        delete h;
        return map_cuda(e);
    }
    char *w = static_cast<char *>(h->ws);
    h->status = reinterpret_cast<int32_t *>(w);
    w += 256;
    for (int32_t **p : {&h->move_src, &h->move_dst, &h->move_cnt}) {
        *p = reinterpret_cast<int32_t *>(w);
        w += (lists + 255) / 256 * 256;
    }
    h->attn = w;
    *out = h;
    return SPECVERIFY_OK;
}

int specverify_tree_destroy(specverify_tree_t h) {
    if (!h) return SPECVERIFY_OK;
    DeviceGuard guard(h->device);
    cudaError_t e = guard.err;
    if (e == cudaSuccess) e = cudaFree(h->ws);
    delete h;
    return map_cuda(e);
}

int specverify_tree_status(specverify_tree_t h, void *cuda_stream, int32_t *status_out) {
    if (!h || !status_out) return SPECVERIFY_ERR_INVALID_ARG;
    DeviceGuard guard(h->device);
    if (guard.err != cudaSuccess) return map_cuda(guard.err);
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    cudaError_t e = cudaMemcpyAsync(status_out, h->status, sizeof(int32_t),
                                    cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(h->status, 0, sizeof(int32_t), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    return map_cuda(e);
}

int specverify_tree_workspace_bytes(specverify_tree_t h, size_t *out) {
    if (!h || !out) return SPECVERIFY_ERR_INVALID_ARG;
    *out = h->ws_bytes;
    return SPECVERIFY_OK;
}

int specverify_tree_set_wait_limit(specverify_tree_t h, uint64_t ns) {
    if (!h) return SPECVERIFY_ERR_INVALID_ARG;
    h->wait_ns = ns == 0 ? sv::kDefaultWaitNs : ns;
    return SPECVERIFY_OK;
}

int specverify_tree_attention(specverify_tree_t h, const specverify_cache *cache,
                              const specverify_tree *tree, const int32_t *lens, const void *q,
                              int64_t rows, int32_t heads, int64_t q_row_stride,
                              int64_t q_head_stride, float scale, void *out,
                              int64_t out_row_stride, int64_t out_head_stride, float *lse,
                              void *cuda_stream) {
    int rc = check_tree(h, tree, false);
    if (rc == SPECVERIFY_OK) rc = check_cache(cache, tree->B, true);
    if (rc == SPECVERIFY_OK) rc = check_rows(cache, q, rows, heads, q_row_stride, q_head_stride);
    if (rc == SPECVERIFY_OK)
        rc = check_rows(cache, out, rows, heads, out_row_stride, out_head_stride);
    if (rc != SPECVERIFY_OK) return rc;
    if (!good_scale(scale)) return SPECVERIFY_ERR_INVALID_ARG;
    // queries may be one row for all, outputs keep to themselves
    const Layout o = rows_layout(rows, heads, cache->head_dim, out_row_stride, out_head_stride);
    if (!o.apart()) return SPECVERIFY_ERR_INVALID_ARG;
    if (tree->B == 0 || rows == 0) return SPECVERIFY_OK;
    if (q == out || (q_row_stride == out_row_stride && q_head_stride == out_head_stride && !o.apart(q, out)))
        return SPECVERIFY_ERR_INVALID_ARG;
    if (!lens) return SPECVERIFY_ERR_INVALID_ARG;
    if (!sv::line_fits((int64_t)cache->max_pages * cache->page_size, cache->kv_heads, sv::kAttnHead,
                       tree->max_nodes, heads / cache->kv_heads))
        return SPECVERIFY_ERR_TOO_LARGE;
    DeviceGuard guard(h->device);
    if (guard.err != cudaSuccess) return map_cuda(guard.err);
    sv::TreeAttnParams p{};
    p.c = cache_params(cache);
    p.t = tree_params(tree);
    p.lens = lens;
    p.q = static_cast<const char *>(q);
    p.q_rs = q_row_stride * 2;
    p.q_hs = q_head_stride * 2;
    p.out = static_cast<char *>(out);
    p.o_rs = out_row_stride * 2;
    p.o_hs = out_head_stride * 2;
    p.lse = lse;
    p.rows = rows;
    p.heads = heads;
    p.G = heads / cache->kv_heads;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.status = h->status;
    p.wait_ns = h->wait_ns;
    sv::attn_place(p, h->attn, h->num_sms);
    return map_cuda(sv::launch_tree_attention(p, h->num_sms,
                                              static_cast<cudaStream_t>(cuda_stream)));
}

int specverify_verify_tree(specverify_tree_t h, const specverify_tree *tree, const void *target,
                           int32_t dtype, int64_t V, int64_t row_stride, int64_t rows,
                           int32_t *n_accepted, int32_t *out_tokens, int32_t *path,
                           void *cuda_stream) {
    const int rc = check_tree(h, tree, true);
    if (rc != SPECVERIFY_OK) return rc;
    if (dtype != SPECVERIFY_FP32 && dtype != SPECVERIFY_BF16) return SPECVERIFY_ERR_INVALID_ARG;
    const int64_t esz = dtype == SPECVERIFY_FP32 ? 4 : 2;
    if (V < 1 || V > INT32_MAX - 64 || row_stride < V || (row_stride * esz) % 16 != 0 || rows < 0)
        return SPECVERIFY_ERR_INVALID_ARG;
    if (tree->B == 0) return SPECVERIFY_OK;
    if ((rows > 0 && (!target || !aligned16(target))) || !n_accepted || !out_tokens || !path)
        return SPECVERIFY_ERR_INVALID_ARG;
    DeviceGuard guard(h->device);
    if (guard.err != cudaSuccess) return map_cuda(guard.err);
    sv::TreeVerifyParams p{};
    p.t = tree_params(tree);
    p.target = static_cast<const char *>(target);
    p.stride_bytes = row_stride * esz;
    p.V = V;
    p.rows = rows;
    p.n_out = n_accepted;
    p.tok_out = out_tokens;
    p.path_out = path;
    p.status = h->status;
    p.wait_ns = h->wait_ns;
    return map_cuda(sv::launch_tree_verify(p, dtype, static_cast<cudaStream_t>(cuda_stream)));
}

int specverify_tree_commit(specverify_tree_t h, const specverify_cache *cache, int32_t B,
                           int32_t max_nodes, const int32_t *lens, const int32_t *seen,
                           const int32_t *n_accepted, const int32_t *path, int32_t *new_lens,
                           int32_t *new_seen, void *cuda_stream) {
    if (!h || B < 0 || B > h->max_batch || max_nodes < 1 || max_nodes > sv::kMaxNodes)
        return SPECVERIFY_ERR_INVALID_ARG;
    const int rc = check_cache(cache, B, false);
    if (rc != SPECVERIFY_OK) return rc;
    if (cache->layers > 65535 || !writable(cache)) return SPECVERIFY_ERR_INVALID_ARG;
    if (B == 0) return SPECVERIFY_OK;
    if (!lens || !n_accepted || !path || !new_lens || (new_seen && !seen) ||
        (cache->pos && !seen))
        return SPECVERIFY_ERR_INVALID_ARG;
    const int64_t n = (int64_t)B * 4;
    const void *in[] = {lens, n_accepted, seen};
    for (const void *a : in)
        if (a && (overlap(a, n, new_lens, n) || (new_seen && overlap(a, n, new_seen, n))))
            return SPECVERIFY_ERR_INVALID_ARG;
    const int64_t np = n * max_nodes;
    if (overlap(path, np, new_lens, n) || (new_seen && overlap(path, np, new_seen, n)) ||
        (new_seen && overlap(new_lens, n, new_seen, n)))
        return SPECVERIFY_ERR_INVALID_ARG;
    DeviceGuard guard(h->device);
    if (guard.err != cudaSuccess) return map_cuda(guard.err);
    sv::CommitParams p{};
    p.c = cache_params(cache);
    p.B = B;
    p.max_nodes = max_nodes;
    p.lens = lens;
    p.seen = seen;
    p.n = n_accepted;
    p.path = path;
    p.new_lens = new_lens;
    p.new_seen = new_seen;
    p.status = h->status;
    return map_cuda(sv::launch_tree_commit(p, static_cast<cudaStream_t>(cuda_stream)));
}

int specverify_cache_accumulate(specverify_tree_t h, const specverify_cache *cache,
                                const specverify_tree *tree, const int32_t *lens,
                                const int32_t *n_accepted, const int32_t *path, const void *q,
                                int64_t rows, int32_t heads, int64_t q_row_stride,
                                int64_t q_head_stride, const float *lse, float scale,
                                void *cuda_stream) {
    int rc = check_tree(h, tree, false);
    if (rc == SPECVERIFY_OK) rc = check_cache(cache, tree->B, true);
    if (rc == SPECVERIFY_OK) rc = check_rows(cache, q, rows, heads, q_row_stride, q_head_stride);
    if (rc != SPECVERIFY_OK) return rc;
    if (!good_scale(scale)) return SPECVERIFY_ERR_INVALID_ARG;
    if (tree->B == 0 || rows == 0) return SPECVERIFY_OK;
    if (!lens || !n_accepted || !path || !lse || !cache->mass || !mass_layout(cache).apart())
        return SPECVERIFY_ERR_INVALID_ARG;
    if (!sv::line_fits((int64_t)cache->max_pages * cache->page_size, cache->kv_heads, sv::kMassHead,
                       tree->max_nodes, heads / cache->kv_heads))
        return SPECVERIFY_ERR_TOO_LARGE;
    DeviceGuard guard(h->device);
    if (guard.err != cudaSuccess) return map_cuda(guard.err);
    sv::AccumParams p{};
    p.c = cache_params(cache);
    p.t = tree_params(tree);
    p.lens = lens;
    p.n = n_accepted;
    p.path = path;
    p.q = static_cast<const char *>(q);
    p.q_rs = q_row_stride * 2;
    p.q_hs = q_head_stride * 2;
    p.lse = lse;
    p.rows = rows;
    p.heads = heads;
    p.G = heads / cache->kv_heads;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.status = h->status;
    p.wait_ns = h->wait_ns;
    return map_cuda(sv::launch_accumulate(p, h->num_sms, static_cast<cudaStream_t>(cuda_stream)));
}

int specverify_cache_evict(specverify_tree_t h, const specverify_cache *cache, int32_t B,
                           const int32_t *lens, const int32_t *seen, int32_t budget, int32_t sink,
                           int32_t recent, float *mass_out, int32_t *pos_out, int32_t *new_lens,
                           void *cuda_stream) {
    if (!h || B < 0 || B > h->max_batch) return SPECVERIFY_ERR_INVALID_ARG;
    const int rc = check_cache(cache, B, false);
    if (rc != SPECVERIFY_OK) return rc;
    if (budget < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > budget)
        return SPECVERIFY_ERR_INVALID_ARG;
    if (B == 0) return SPECVERIFY_OK;
    if (!cache->mass || !cache->pos || !lens || !seen || !mass_out || !pos_out || !new_lens ||
        !writable(cache))
        return SPECVERIFY_ERR_INVALID_ARG;
    const Layout m = mass_layout(cache);
    if ((mass_out != cache->mass && !m.apart(mass_out, cache->mass)) ||
        (pos_out != cache->pos && !m.apart(pos_out, cache->pos)) || !m.apart(mass_out, pos_out) ||
        !m.apart(mass_out, cache->pos) || !m.apart(pos_out, cache->mass))
        return SPECVERIFY_ERR_INVALID_ARG;
    const int64_t n = (int64_t)B * 4;
    if (overlap(lens, n, new_lens, n) || overlap(seen, n, new_lens, n))
        return SPECVERIFY_ERR_INVALID_ARG;
    const int64_t items = (int64_t)cache->layers * B * cache->kv_heads;
    const int64_t capacity = (int64_t)cache->max_pages * cache->page_size;
    const int64_t moves = budget < capacity ? std::min((int64_t)budget, capacity - budget) : 0;
    if (items > INT32_MAX || items * moves > h->max_moves) return SPECVERIFY_ERR_TOO_LARGE;
    DeviceGuard guard(h->device);
    if (guard.err != cudaSuccess) return map_cuda(guard.err);
    sv::EvictParams p{};
    p.c = cache_params(cache);
    p.B = B;
    p.lens = lens;
    p.seen = seen;
    p.budget = budget;
    p.sink = sink;
    p.recent = recent;
    p.mass_out = mass_out;
    p.pos_out = pos_out;
    p.new_lens = new_lens;
    p.moves = (int32_t)moves;
    p.move_src = h->move_src;
    p.move_dst = h->move_dst;
    p.move_cnt = h->move_cnt;
    p.status = h->status;
    return map_cuda(sv::launch_evict(p, static_cast<cudaStream_t>(cuda_stream)));
}

}  // extern "C"
