// paged.cuh -- the paged KV cache: what its page calls and its attention kernels share.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/vc.h"

namespace vc {

// vc_paged_kv as the kernels take it (one layer's pages for attention, every layer's for page calls)
struct PagedKv {
    uint16_t *k, *v;
    int *table, *len, *refs, *status;
    int layers, pages, page, page_shift, Hk, Dh, Hq, seqs, columns, window, sinks;
};

struct PagedWorkspace {
    int* head;        // [0] copies listed by a resize or fork, [1], [2] a compaction's moves and live pages, [3] rows to clear
    int* ticket;      // work handed out by attention (zero between calls)
    int* merge;       // arrival counters of split attention work [kMaxSplitCtas] (zero between calls)
    int* copies;      // [seqs][3]: source page, destination page, positions to copy
    int* ok;          // [seqs]: rows of a fork that are done, of a step whose sessions start anew
    int* first;       // [seqs]: the lowest row that names a session
    int4* rows;       // [seqs]: a resize's rows
    int* need;        // [seqs][2]: a row's first page request and how many it has
    int* chunk_live;  // compaction: pages in use per chunk of kCompactChunk
    int* rename;      // [pages]: resize and fork: the free pages to hand out; compact: a page's move, -1: none
    int* moves;       // [pages][2]: source and destination of each move of a compaction
    float* partial;   // split attention work
    size_t bytes;
};

static constexpr int kMaxSms = 256;
static constexpr int kCompactChunk = 4096;
static constexpr int kMaxSplitCtas = 2 * kMaxSms;      // CTAs of an attention launch that splits the key axis
// rows of the records that split attention work leaves: kMaxSplitCtas tiles of 64 or 128 rows, or kMaxSms of the
// prompts' tiles (512 rows of 64 dimensions, 256 of 128)
static constexpr int kRecordRows = 512 * kMaxSms / 2, kRecordRows64 = 512 * kMaxSms;

// the workspace's parts, in order; false where the sizes are outside the documented limits
bool paged_sizes_ok(const vc_paged_kv& c);
PagedWorkspace paged_carve(const vc_paged_kv& c, void* base);
// sizes, pointers and workspace as documented
bool paged_kv_ok(const vc_paged_kv* c);
PagedKv paged_kernel_kv(const vc_paged_kv& c);

struct PagedAttnArgs {
    PagedKv c;                   // k, v: this layer's
    const uint16_t *q, *kn, *vn; // new rows
    uint16_t* out;
    long long q_ld, k_ld, v_ld, out_ld;
    const int *seqs, *pos, *cu_rows;
    int batch, rows, f16, num_sms;
    int pdl;                     // 1: launches may begin while the one before ends (programmatic dependent launch)
    int widen;                   // store bf16 results in fp16's format (the input of a quantized projection)
    float scale_log2;            // scale * log2(e)
    int* merge;
    int* ticket;                 // counts the pieces handed out (zero between calls)
    float* partial;
};

// appends and attends for one layer: the form by the rows' kind (one per session, or prompts) and the shape.  The
// caller fills in the rows and the scale, this call the cache, its workspace and the device.
cudaError_t paged_attend(const vc_paged_kv& kv, int layer, PagedAttnArgs a, cudaStream_t s);

// rows of a fused projection [q | k | v] of ld elements a row, 1 / sqrt(Dh), results of out_ld elements a row
PagedAttnArgs paged_rows(const uint16_t* qkv, int ld, int Hq, int Hk, int Dh, uint16_t* out, int out_ld, int widen, int pdl);

// joins the records of tiles of attention whose key blocks were split over CTAs
struct JoinShape {
    int rows, tile_rows;     // of a record; packed rows of a tile (tiles of prompts hold whole tokens)
    int keys;                // of a block
    int most_tiles, ctas;    // as the launch before was given them
};
// whether a row may see so many keys that joins take a launch of their own.  (8 heads of 64 over 32, 30 rows behind 30000
// positions: 57 us for 73; 4 sessions of 2 rows behind 107: 17.7 for 12.0)
inline bool many_keys(const PagedAttnArgs& a) {
    return (a.c.window > 0 ? (long long)a.c.window + a.c.sinks + a.rows : (long long)a.c.columns * a.c.page) > 8192;
}
cudaError_t launch_paged_join(const PagedAttnArgs& a, const JoinShape& w, cudaStream_t s);
cudaError_t launch_paged_append(const PagedAttnArgs& a, cudaStream_t s);
cudaError_t launch_paged_tiles(const PagedAttnArgs& a, cudaStream_t s);
// the tensor-core form for many rows; cudaErrorNotSupported: the shape is not covered
cudaError_t launch_paged_prompts(const PagedAttnArgs& a, cudaStream_t s);
// one row per session, appended and attended in one launch; cudaErrorNotSupported: the shape is not covered
cudaError_t launch_paged_frames(const PagedAttnArgs& a, cudaStream_t s);

// the state that a backbone keeps beside the pages: frames of each session, and dense parts (frames among them)
struct PagedFrames {
    const int* count;
    vc_session_part parts[3];
    int n_parts;
};
// frames: null, or a backbone's step: a session that starts at position 0 with frames behind it (it was ended) starts anew,
// its parts zero; one that holds another number of positions than frames is a bad row
cudaError_t launch_paged_resize(const PagedKv& c, const PagedWorkspace& w, int n, const int* seqs, const int* lens,
                                int add, int* pos, int pdl, cudaStream_t s, const PagedFrames* frames = nullptr);
cudaError_t launch_paged_fork(const PagedKv& c, const PagedWorkspace& w, int n, const int* src, const int* dst,
                              const vc_session_part* parts, int n_parts, int* done, cudaStream_t s);
cudaError_t launch_paged_compact(const PagedKv& c, const PagedWorkspace& w, int* live, cudaStream_t s);

}  // namespace vc
