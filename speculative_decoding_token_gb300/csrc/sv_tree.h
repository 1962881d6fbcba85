// sv_tree.h -- types shared by the host library and the kernels of the
// token-tree calls (not part of the public C ABI).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "specverify.h"

namespace sv {

constexpr int kMaxNodes = SPECVERIFY_MAX_NODES;
constexpr int kMaskWords = kMaxNodes / 32;
constexpr int kTileSlots = 128;  // slots of a tile of keys

// An item's place on the work line of attention or accumulation starts with that
// many units that are no tiles (what a start costs: see the kernels).
constexpr int kAttnHead = 6, kMassHead = 1;

// Whether the kernels' 31-bit counts hold: units of a sequence's key heads on the
// line, and rows (nodes times the heads of a key head) of an item.
inline bool line_fits(int64_t slots, int64_t kv_heads, int head, int64_t nodes, int64_t group) {
    return ((slots + kTileSlots - 1) / kTileSlots + head) * kv_heads <= INT32_MAX &&
           nodes * group <= INT32_MAX - 2 * kTileSlots;
}

// A paged cache, strides in bytes.
struct CacheParams {
    char *k, *v;
    int64_t ls, ps, hs, ts;   // layer, page, head, token strides
    float *mass;
    int32_t *pos;
    int64_t mls, mps, mhs, mts;  // of mass and pos, elements
    const int32_t *table;
    int64_t table_stride;
    int64_t num_pages;
    int32_t max_pages, page, kv_heads, d, layers;
    int32_t fp16;             // 1: binary16, 0: bfloat16
    // s / page for 0 <= s < 2^31: the high word of s * page_mul, shifted right
    // (Granlund and Montgomery, "Division by invariant integers using
    // multiplication", with 2^(31 + l) / page rounded up, 2^l >= page)
    uint32_t page_mul;
    int32_t page_shift;
};

inline void set_page(CacheParams &c, int32_t page) {
    int l = 0;
    while (((int64_t)1 << l) < page) ++l;
    c.page = page;
    c.page_mul = (uint32_t)(((uint64_t)1 << (31 + l)) / (uint32_t)page + 1);
    c.page_shift = l - 1;
}

struct TreeParams {
    const int64_t *row_off;
    const int32_t *nodes, *parent, *tokens;
    int32_t B, max_nodes;
};

struct TreeAttnParams {
    CacheParams c;
    TreeParams t;
    const int32_t *lens;
    const char *q;
    int64_t q_rs, q_hs;       // bytes
    char *out;
    int64_t o_rs, o_hs;       // bytes
    float *lse;
    int64_t rows;
    int32_t heads, G;
    float scale_log2;         // scale * log2(e)
    int32_t box;              // tokens of one tiled copy: divides the page size and a tile
    int32_t blocks;           // blocks of 256 rows that a tree can have
    int32_t *status;
    uint64_t wait_ns;         // bound of a wait inside the kernel
    // workspace: the pieces of rows whose slots were split over CTAs
    float *piece_o;           // [CTAs, 2, 256, d]
    float2 *piece_ml;         // [CTAs, 2, 256]: reference maximum (log2 scale), sum
    struct AttnOwner *owner;  // [CTAs]
};

// The item that a CTA begins and another ends.
struct AttnOwner {
    int64_t row0;             // its tree's first row
    int32_t pieces;           // 0: there is none
    int32_t rows, first_row;  // of the item, and its first among the tree's rows of a key head
    int32_t head;             // key head
};

struct TreeVerifyParams {
    TreeParams t;
    const char *target;
    int64_t stride_bytes, V, rows;
    int32_t *n_out, *tok_out, *path_out;
    int32_t *status;
    uint64_t wait_ns;
};

struct CommitParams {
    CacheParams c;
    int32_t B, max_nodes;
    const int32_t *lens, *seen, *n, *path;
    int32_t *new_lens, *new_seen;
    int32_t *status;
};

struct AccumParams {
    CacheParams c;
    TreeParams t;
    const int32_t *lens, *n, *path;
    const char *q;
    int64_t q_rs, q_hs;
    const float *lse;
    int64_t rows;
    int32_t heads, G;
    float scale_log2;
    int32_t box;              // as of the attention
    int32_t *status;
    uint64_t wait_ns;
};

struct EvictParams {
    CacheParams c;
    int32_t B;
    const int32_t *lens, *seen;
    int32_t budget, sink, recent;
    float *mass_out;
    int32_t *pos_out, *new_lens;
    int32_t moves;            // list entries of one item: min(budget, capacity - budget)
    int32_t *move_src, *move_dst;  // [items, moves]
    int32_t *move_cnt;        // [items]
    int32_t inline_moves;     // the selecting CTA makes its item's moves
    int32_t *status;
};

cudaError_t prepare_tree();
size_t attn_workspace(int ctas);
void attn_place(TreeAttnParams &p, void *ws, int ctas);
cudaError_t launch_tree_attention(TreeAttnParams p, int num_sms, cudaStream_t s);
cudaError_t launch_tree_verify(const TreeVerifyParams &p, int dtype, cudaStream_t s);
cudaError_t launch_tree_commit(const CommitParams &p, cudaStream_t s);
cudaError_t prepare_accumulate();
cudaError_t launch_accumulate(AccumParams p, int num_sms, cudaStream_t s);
cudaError_t prepare_evict();
cudaError_t launch_evict(EvictParams p, cudaStream_t s);

#ifdef __CUDACC__
// A launch that may begin while the stream's kernel before it ends (programmatic
// dependent launch): the kernel sets itself up and then waits for what came
// before with after_previous(), ahead of its first access to global memory, in
// every CTA. A step is a row of short kernels, and this hides their starts.
template <class Kernel, class... Args>
cudaError_t launch_after(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t s,
                         int cluster, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---------------------------------------------------------------------------
// device helpers

// A line of work units cut over CTAs: CTA i has units [cut.at(i), cut.at(i + 1)),
// at(i) = floor(i total / ctas), so that halves of the line are halves of the CTAs.
struct Cut {
    int ctas, more;
    long long each;

    __device__ __forceinline__ Cut(long long total, int grid) {
        ctas = (int)min((long long)grid, total);
        if (ctas == 0) ctas = 1;  // no units: they all are CTA 0's
        each = total >> 31 ? total / ctas : (long long)((int)total / ctas);
        more = (int)(total - each * ctas);
    }
    __device__ __forceinline__ long long at(int i) const { return i * each + i * more / ctas; }
    // The CTA of a unit.
    __device__ __forceinline__ int of(long long unit) const {
        int i = 0;  // at(i) <= unit < at(i + 1), by halves
        for (int step = 1 << (31 - __clz(ctas)); step > 0; step >>= 1)
            if (i + step < ctas && at(i + step) <= unit) i += step;
        return i;
    }
};

// Waits until the kernels before this one are done and their writes are seen,
// then lets the next one set itself up.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

// Whether tokens [0, count) of sequence b fit its pages.
__device__ __forceinline__ bool cache_holds(const CacheParams &c, int64_t count) {
    return count >= 0 && count <= (int64_t)c.max_pages * c.page;
}

// Page i of sequence b, -1 for an id outside the pool.
__device__ __forceinline__ int64_t page_at(const CacheParams &c, int b, int i) {
    const int32_t id = c.table[(int64_t)b * c.table_stride + i];
    return id >= 0 && (int64_t)id < c.num_pages ? (int64_t)id : -1;
}

// Slot s's place: page `index` of its sequence, token `token` of that page.
struct Place {
    int index, token;
};

__device__ __forceinline__ Place place_of(const CacheParams &c, int s) {
    const int i = (int)(__umulhi((uint32_t)s, c.page_mul) >> c.page_shift);
    return {i, s - i * c.page};
}

// The page that holds slot s of sequence b.
__device__ __forceinline__ int64_t page_of(const CacheParams &c, int b, int s) {
    return page_at(c, b, place_of(c, s).index);
}

#endif

}  // namespace sv
