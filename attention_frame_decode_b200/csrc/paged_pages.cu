// paged_pages.cu -- the page calls of the paged KV cache: resize, fork and compact.
//
// The bookkeeping is a chain of small steps over the sessions' rows (who releases what, who needs how many
// pages, which free pages they get), each of which needs the one before for all rows: one CTA takes them in
// turn with block barriers, so that a call is one launch for the tables and one for the data.  Every result
// is a function of the inputs alone: releases are counted before anything is taken, requests are numbered by
// a prefix sum in row order, and the k-th request gets the k-th lowest free page.
#include "common.cuh"
#include "paged.cuh"

namespace vc {

static constexpr int kPT = 1024;   // threads of a bookkeeping CTA

VC_DEV int ceil_pages(int positions, int shift, int page) { return (positions + page - 1) >> shift; }

// exclusive prefix sum over the CTA's threads; `total` gets the sum (all threads call; two barriers)
VC_DEV int block_scan(int v, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int w = lane < nw ? warp_sums[lane] : 0, wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, wi, o);
        if (lane >= o) wi += u;
    }
    total = __shfl_sync(0xffffffffu, wi, 31);
    const int before = __shfl_sync(0xffffffffu, wi - w, warp);
    __syncthreads();
    return before + incl - v;
}

// the lowest `want` free pages in ascending order into list; returns how many there are (all threads call)
VC_DEV int find_free(const int* refs, int pages, int want, int* list, int* warp_sums) {
    constexpr int PER = 16;
    int found = 0;
    for (int base = 0; base < pages && found < want; base += kPT * PER) {
        const int p0 = base + (int)threadIdx.x * PER;
        unsigned free_bits = 0;
#pragma unroll
        for (int q = 0; q < PER / 4; ++q) {
            const int p = p0 + 4 * q;
            if (p + 4 <= pages) {
                const int4 r = __ldcg(reinterpret_cast<const int4*>(refs + p));
                free_bits |= ((r.x <= 0 ? 1u : 0u) | (r.y <= 0 ? 2u : 0u) | (r.z <= 0 ? 4u : 0u) | (r.w <= 0 ? 8u : 0u)) << (4 * q);
            } else {
                for (int u = 0; u < 4; ++u)
                    if (p + u < pages && __ldcg(refs + p + u) <= 0) free_bits |= 1u << (4 * q + u);
            }
        }
        int total;
        int at = found + block_scan(__popc(free_bits), warp_sums, total);
        while (free_bits && at < want) {
            const int b = __ffs(free_bits) - 1;
            free_bits &= free_bits - 1;
            list[at++] = p0 + b;
        }
        found += total;
    }
    return min(found, want);
}

// the threads that take a row together: a warp, or where there are many rows half or a quarter of one (the rows' chains of
// loads run beside one another: a turn of 512 sessions that takes 6234 pages: 33 us with a warp each, 30 with a quarter)
struct Team {
    int index, lane, size, count;   // this team, this thread in it, threads of a team, teams of the CTA
    unsigned mask;                  // its lanes of the warp
};
VC_DEV Team team_for(int rows) {
    Team t;
    t.size = rows <= 32 ? 32 : rows <= 64 ? 16 : 8;
    t.index = (int)threadIdx.x / t.size;
    t.lane = (int)threadIdx.x & (t.size - 1);
    t.count = kPT / t.size;
    t.mask = t.size == 32 ? 0xffffffffu : ((1u << t.size) - 1u) << (threadIdx.x & 31 & ~(t.size - 1));
    return t;
}

// takes the team's session row of the table: releases the mapped entries of columns [c0, c1)
VC_DEV void release_columns(const PagedKv& c, int* row, int c0, int c1, const Team& t) {
    for (int at = c0 + t.lane; at < c1; at += 4 * t.size) {
        int e[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) e[u] = at + u * t.size < c1 ? row[at + u * t.size] : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if ((unsigned)e[u] < (unsigned)c.pages) atomicSub(c.refs + e[u], 1);
            if (at + u * t.size < c1) row[at + u * t.size] = -1;
        }
    }
}

// marks each row that names a session (in range) first: first[s] = the lowest row that names it
VC_DEV void mark_first(const int* idx, int n, int seqs, int* first) {
    for (int i = threadIdx.x; i < n; i += kPT)
        if ((unsigned)idx[i] < (unsigned)seqs) first[idx[i]] = INT32_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPT)
        if ((unsigned)idx[i] < (unsigned)seqs) atomicMin(first + idx[i], i);
    __syncthreads();
}

// ------------------------------------------------------------------------------------------
// resize
// ------------------------------------------------------------------------------------------
// a row's session (< 0: the row is bad), its length, the length asked for (INT32_MAX: more than the columns hold)
VC_DEV int4 resize_row(const PagedKv& c, const int* seqs, const int* lens, int add, const int* first, int i, const int* frames) {
    int4 r = make_int4(-1, 0, 0, 0);
    const int s = seqs ? seqs[i] : i, most = c.columns << c.page_shift;
    if ((unsigned)s >= (unsigned)c.seqs || (seqs && __ldcg(first + s) != i)) return r;
    const int have = c.len[s];
    const long long to = (long long)(lens ? lens[i] : have) + add;
    if (to < 0 || have < 0 || have > most) return r;
    if (frames && have > 0 && frames[s] != have) return r;   // its recurrent state belongs to another position
    r.y = have;
    r.z = to <= most ? (int)to : INT32_MAX;
    // the page that is written next has to be there (it is not where a length ends in positions given up)
    const int at = min(r.y, r.z);
    if ((at & (c.page - 1)) && (unsigned)c.table[(size_t)s * c.columns + (at >> c.page_shift)] >= (unsigned)c.pages)
        return r;
    r.x = s;
    return r;
}

__global__ void __launch_bounds__(kPT) paged_resize_kernel(const PagedKv c, const PagedWorkspace w, int n,
                                                           const int* seqs, const int* lens, int add, int* pos,
                                                           const int* frames) {
    __shared__ int warp_sums[32];
    __shared__ int copies, anew;
    const int tid = threadIdx.x;
    pdl_trigger();
    if (seqs) mark_first(seqs, n, c.seqs, w.first);
    for (int i = tid; i < n; i += kPT) w.rows[i] = resize_row(c, seqs, lens, add, w.first, i, frames);
    __syncthreads();

    // 1. releases
    const Team team = team_for(n);
    for (int i = team.index; i < n; i += team.count) {
        const int4 r = w.rows[i];
        const int s = r.x, have = r.y, to = r.z;
        if (s < 0) continue;
        int* row = c.table + (size_t)s * c.columns;
        if (to < have)
            release_columns(c, row, ceil_pages(to, c.page_shift, c.page), ceil_pages(have, c.page_shift, c.page), team);
        if (c.window > 0) {
            // columns behind the sinks whose last position is at most start - window; those below an unmapped one
            // were released by an earlier call
            const int start = min(to, have);
            const int lo = (int)(((long long)c.sinks + c.page - 1) >> c.page_shift);
            int hi = start - c.window + 1 > 0 ? (start - c.window + 1) >> c.page_shift : 0;
            while (hi > lo) {
                const int col = hi - 1 - team.lane;
                int e = -1;
                if (col >= lo) {
                    e = row[col];
                    if ((unsigned)e < (unsigned)c.pages) {
                        atomicSub(c.refs + e, 1);
                        row[col] = -1;
                    } else e = -1;
                }
                if (__any_sync(team.mask, e < 0)) break;
                hi -= team.size;
            }
        }
    }
    if (tid == 0) copies = anew = 0;
    __syncthreads();

    // 2. requests, numbered in row order; w.need[i]: the row's first request, w.need[n + i]: how many
    int asked = 0;
    for (int base = 0; base < n; base += kPT) {
        const int i = base + tid;
        int need = 0;
        if (i < n) {
            const int4 r = w.rows[i];
            const int s = r.x, have = r.y, to = r.z;
            if (s >= 0 && to > have && to != INT32_MAX) {
                need = ceil_pages(to, c.page_shift, c.page) - ceil_pages(have, c.page_shift, c.page);
                if ((have & (c.page - 1)) && __ldcg(c.refs + c.table[(size_t)s * c.columns + (have >> c.page_shift)]) > 1)
                    need++;
            }
        }
        int total;
        const int at = asked + block_scan(need, warp_sums, total);
        if (i < n) {
            w.need[2 * i] = at;
            w.need[2 * i + 1] = need;
        }
        asked += total;
    }
    const int found = asked ? find_free(c.refs, c.pages, min(asked, c.pages), w.rename, warp_sums) : 0;
    __syncthreads();

    // 3. pages, lengths, positions
    for (int i = team.index; i < n; i += team.count) {
        const int4 r = w.rows[i];
        const int s = r.x, have = r.y, to = r.z;
        const int at = w.need[2 * i], need = w.need[2 * i + 1];
        const bool granted = s >= 0 && to != INT32_MAX && (need == 0 || need <= found - at);
        if (granted && need) {
            int* row = c.table + (size_t)s * c.columns;
            const int c0 = ceil_pages(to, c.page_shift, c.page) - need;   // the request's first column
            for (int q0 = team.lane; q0 < need; q0 += 4 * team.size) {
                int page[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) page[u] = q0 + u * team.size < need ? w.rename[at + q0 + u * team.size] : 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int q = q0 + u * team.size, col = c0 + q;
                    if (q >= need) break;
                    if (col < ceil_pages(have, c.page_shift, c.page)) {   // a shared page's copy
                        const int old = row[col];
                        atomicSub(c.refs + old, 1);
                        const int k = atomicAdd(&copies, 1);
                        w.copies[3 * k] = old;
                        w.copies[3 * k + 1] = page[u];
                        w.copies[3 * k + 2] = have & (c.page - 1);
                    }
                    row[col] = page[u];
                    c.refs[page[u]] = 1;
                }
            }
        }
        if (team.lane == 0) {
            if (granted) c.len[s] = to;
            if (pos) pos[i] = granted ? min(have, to) : -1;
            if (!granted) atomicOr(c.status, s < 0 ? VC_DEV_INVALID : VC_DEV_CAPACITY);
            if (frames) {   // a step's session that was ended
                w.ok[i] = granted && have == 0 && frames[s] != 0;
                if (w.ok[i]) atomicAdd(&anew, 1);
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        w.head[0] = copies;
        w.head[3] = anew;
    }
}

// ------------------------------------------------------------------------------------------
// fork
// ------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kPT) paged_fork_kernel(const PagedKv c, const PagedWorkspace w, int n, const int* src,
                                                         const int* dst, int* done) {
    __shared__ int warp_sums[32];
    __shared__ int copies;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    // first[s]: the lowest row that forks onto s, -1 where a row forks from s
    mark_first(dst, n, c.seqs, w.first);
    for (int i = tid; i < n; i += kPT)
        if ((unsigned)src[i] < (unsigned)c.seqs) w.first[src[i]] = -1;
    if (tid == 0) copies = 0;
    __syncthreads();
    auto good = [&](int i) {
        return (unsigned)src[i] < (unsigned)c.seqs && (unsigned)dst[i] < (unsigned)c.seqs && __ldcg(w.first + dst[i]) == i;
    };
    // 1. what the destinations hold goes back
    const Team whole_warp = team_for(1);
    for (int i = warp; i < n; i += kPT / 32) {
        if (!good(i)) continue;
        const int have = min(max(c.len[dst[i]], 0), c.columns << c.page_shift);
        release_columns(c, c.table + (size_t)dst[i] * c.columns, 0, ceil_pages(have, c.page_shift, c.page), whole_warp);
    }
    __syncthreads();
    // 2. a page for each partly filled last one, numbered in row order
    int asked = 0;
    for (int base = 0; base < n; base += kPT) {
        const int i = base + tid;
        int need = 0;
        if (i < n && good(i)) {
            const int have = min(max(c.len[src[i]], 0), c.columns << c.page_shift);
            if (have & (c.page - 1)) {
                const int e = c.table[(size_t)src[i] * c.columns + (have >> c.page_shift)];
                need = (unsigned)e < (unsigned)c.pages ? 1 : 0;
            }
        }
        int total;
        const int at = asked + block_scan(need, warp_sums, total);
        if (i < n) {
            w.need[2 * i] = at;
            w.need[2 * i + 1] = need;
        }
        asked += total;
    }
    const int found = asked ? find_free(c.refs, c.pages, min(asked, c.pages), w.rename, warp_sums) : 0;
    __syncthreads();
    // 3. shared pages and lengths
    for (int i = warp; i < n; i += kPT / 32) {
        const bool ok = good(i);
        const int at = w.need[2 * i], need = w.need[2 * i + 1];
        const bool granted = ok && (need == 0 || at < found);
        if (granted) {
            const int* theirs = c.table + (size_t)src[i] * c.columns;
            int* mine = c.table + (size_t)dst[i] * c.columns;
            const int have = min(max(c.len[src[i]], 0), c.columns << c.page_shift), whole = have >> c.page_shift;
            for (int col = lane; col < whole; col += 32) {
                const int e = theirs[col];
                if ((unsigned)e >= (unsigned)c.pages) continue;
                mine[col] = e;
                atomicAdd(c.refs + e, 1);
            }
            if (lane == 0) {
                if (need) {
                    const int page = w.rename[at];
                    mine[whole] = page;
                    c.refs[page] = 1;
                    const int k = atomicAdd(&copies, 1);
                    w.copies[3 * k] = theirs[whole];
                    w.copies[3 * k + 1] = page;
                    w.copies[3 * k + 2] = have & (c.page - 1);
                }
                c.len[dst[i]] = have;
            }
        }
        if (lane == 0) {
            if (ok && !granted) c.len[dst[i]] = 0;
            if (!granted) atomicOr(c.status, ok ? VC_DEV_CAPACITY : VC_DEV_INVALID);
            w.ok[i] = granted;
            if (done) done[i] = granted;
        }
        __syncwarp();
    }
    __syncthreads();
    if (tid == 0) w.head[0] = copies;
}

// ------------------------------------------------------------------------------------------
// copies: the listed pages' first positions in every layer, and the sessions' dense state.  A CTA takes one
// item at a time: a head's rows of one page (contiguous), or 32 KB of one session's state; every thread has
// eight 16-byte loads in flight before it stores.  Bound: HBM.
// ------------------------------------------------------------------------------------------
static constexpr int kCopyThreads = 256, kCopyChunk = kCopyThreads * 16 * 8;

struct CopyParts {
    vc_session_part p[8];
    int n;
};

VC_DEV void copy_bytes16(uint8_t* to, const uint8_t* from, int bytes) {
    for (int b0 = threadIdx.x * 16; b0 < bytes; b0 += kCopyChunk) {
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (b0 + u * kCopyThreads * 16 < bytes) v[u] = *reinterpret_cast<const uint4*>(from + b0 + u * kCopyThreads * 16);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (b0 + u * kCopyThreads * 16 < bytes) *reinterpret_cast<uint4*>(to + b0 + u * kCopyThreads * 16) = v[u];
    }
}

// bytes of one session (a multiple of 4) to zero, by the whole grid
VC_DEV void clear_bytes(uint8_t* to, long long bytes, bool wide) {
    const long long first = ((long long)blockIdx.x * kCopyThreads + threadIdx.x) * 16, step = (long long)gridDim.x * kCopyThreads * 16;
    for (long long b = first; b < bytes; b += step) {
        if (wide) *reinterpret_cast<uint4*>(to + b) = make_uint4(0u, 0u, 0u, 0u);
        else
            for (int q = 0; q < 16 && b + q < bytes; q += 4) *reinterpret_cast<uint32_t*>(to + b + q) = 0u;
    }
}

// src null: a step's sessions (dst, null: row i is session i) that start anew have their parts cleared
__global__ void __launch_bounds__(kCopyThreads) paged_copy_kernel(const PagedKv c, const PagedWorkspace w, int n,
                                                                  const int* src, const int* dst, const CopyParts parts) {
    pdl_wait();
    const int per = c.layers * 2 * c.Hk;
    const long long page_items = (long long)w.head[0] * per;
    for (long long it = blockIdx.x; it < page_items; it += gridDim.x) {
        const int* cp = w.copies + 3 * (it / per);
        const int u = (int)(it % per), j = u % c.Hk, layer = u / c.Hk >> 1;
        uint16_t* pool = ((u / c.Hk) & 1) ? c.v : c.k;
        const size_t from = (((size_t)layer * c.pages + cp[0]) * c.Hk + j) * c.page * c.Dh;
        const size_t to = (((size_t)layer * c.pages + cp[1]) * c.Hk + j) * c.page * c.Dh;
        copy_bytes16((uint8_t*)(pool + to), (const uint8_t*)(pool + from), cp[2] * c.Dh * 2);
    }
    if (!src) {
        if (parts.n == 0 || w.head[3] == 0) return;
        for (int i = 0; i < n; ++i) {
            if (!w.ok[i]) continue;
            for (int k = 0; k < parts.n; ++k) {
                const vc_session_part& p = parts.p[k];
                uint8_t* mine = (uint8_t*)p.base + (long long)(dst ? dst[i] : i) * p.stride;
                const bool wide = (((uintptr_t)p.base | p.bytes | p.stride | p.outer_stride) & 15) == 0;
                for (int o = 0; o < p.outer; ++o) clear_bytes(mine + o * p.outer_stride, p.bytes, wide);
            }
        }
        return;
    }
    for (int k = 0; k < parts.n; ++k) {
        const vc_session_part& p = parts.p[k];
        const bool wide = ((p.bytes | p.stride | p.outer_stride) & 15) == 0;
        const long long chunks = (p.bytes + kCopyChunk - 1) / kCopyChunk;
        const long long items = chunks * p.outer * n;
        for (long long it = blockIdx.x; it < items; it += gridDim.x) {
            const int i = (int)(it / (chunks * p.outer));
            if (!w.ok[i]) continue;
            const long long rem = it % (chunks * p.outer), o = rem / chunks, b = rem % chunks * kCopyChunk;
            uint8_t* block = (uint8_t*)p.base + o * p.outer_stride + b;
            const int bytes = (int)(p.bytes - b < kCopyChunk ? p.bytes - b : kCopyChunk);
            const uint8_t* from = block + (long long)src[i] * p.stride;
            uint8_t* to = block + (long long)dst[i] * p.stride;
            if (wide) copy_bytes16(to, from, bytes);
            else
                for (int q = threadIdx.x * 4; q < bytes; q += kCopyThreads * 4)
                    *reinterpret_cast<uint32_t*>(to + q) = *reinterpret_cast<const uint32_t*>(from + q);
        }
    }
}

// ------------------------------------------------------------------------------------------
// compact: live pages are counted per chunk, then listed with the holes that take them, then moved.
// ------------------------------------------------------------------------------------------
static constexpr int kCT = 256;

__global__ void __launch_bounds__(kCT) paged_count_kernel(const PagedKv c, const PagedWorkspace w) {
    __shared__ int warp_sums[32];
    pdl_trigger();
    int live = 0;
    for (int u = 0; u < kCompactChunk / kCT; ++u) {
        const int p = blockIdx.x * kCompactChunk + u * kCT + (int)threadIdx.x;
        live += p < c.pages && c.refs[p] > 0;
    }
    int total;
    block_scan(live, warp_sums, total);
    if (threadIdx.x == 0) w.chunk_live[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kCT) paged_list_kernel(const PagedKv c, const PagedWorkspace w, int* live_out) {
    __shared__ int warp_sums[32];
    pdl_trigger();
    pdl_wait();
    // N pages are live: `before` of them in earlier chunks, `low` of them already below N
    int all = 0, mine = 0;
    for (int k = threadIdx.x; k < (int)gridDim.x; k += kCT) {
        all += w.chunk_live[k];
        mine += k < (int)blockIdx.x ? w.chunk_live[k] : 0;
    }
    int N, before, low;
    block_scan(all, warp_sums, N);
    block_scan(mine, warp_sums, before);
    const int edge = N / kCompactChunk;   // the chunk that N cuts
    int under = 0;
    for (int k = threadIdx.x; k < edge; k += kCT) under += w.chunk_live[k];
    for (int p = edge * kCompactChunk + (int)threadIdx.x; p < N; p += kCT) under += c.refs[p] > 0;
    block_scan(under, warp_sums, low);
    constexpr int PER = kCompactChunk / kCT;
    const int p0 = blockIdx.x * kCompactChunk + (int)threadIdx.x * PER;
    unsigned bits = 0;
    for (int u = 0; u < PER; ++u)
        if (p0 + u < c.pages && c.refs[p0 + u] > 0) bits |= 1u << u;
    int total;
    int lp = before + block_scan(__popc(bits), warp_sums, total);
    for (int u = 0; u < PER; ++u) {
        const int p = p0 + u;
        if (p >= c.pages) break;
        const bool is_live = (bits >> u) & 1u;
        const int k = lp - low;
        w.rename[p] = is_live && p >= N ? k : -1;
        if (is_live && p >= N) w.moves[2 * k] = p;
        if (!is_live && p < N) w.moves[2 * (p - lp) + 1] = p;
        lp += is_live;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        w.head[1] = N - low;
        w.head[2] = N;
        if (live_out) *live_out = N;
    }
}

__global__ void __launch_bounds__(kCopyThreads) paged_move_kernel(const PagedKv c, const PagedWorkspace w) {
    pdl_wait();
    const int moves = w.head[1], N = w.head[2];
    for (int k = blockIdx.x * kCopyThreads + (int)threadIdx.x; k < moves; k += gridDim.x * kCopyThreads) {
        const int from = w.moves[2 * k], to = w.moves[2 * k + 1];
        c.refs[to] = c.refs[from];
        c.refs[from] = 0;
    }
    for (int s = blockIdx.x; s < c.seqs; s += gridDim.x) {
        int* row = c.table + (size_t)s * c.columns;
        const int cols = ceil_pages(min(max(c.len[s], 0), c.columns << c.page_shift), c.page_shift, c.page);
        for (int col = threadIdx.x; col < cols; col += kCopyThreads) {
            const int e = row[col];
            if (e < N || e >= c.pages) continue;
            const int k = w.rename[e];
            if (k >= 0) row[col] = w.moves[2 * k + 1];
        }
    }
    const size_t page_bytes = (size_t)c.Hk * c.page * c.Dh * 2;
    const long long chunks = (long long)((page_bytes + kCopyChunk - 1) / kCopyChunk), per = chunks * 2 * c.layers;
    for (long long it = blockIdx.x; it < per * moves; it += gridDim.x) {
        const int k = (int)(it / per), u = (int)(it % per), layer = (int)(u / chunks) >> 1;
        const size_t b = (size_t)(u % chunks) * kCopyChunk;
        uint8_t* pool = (uint8_t*)(((u / chunks) & 1) ? c.v : c.k) + b;
        const size_t from = ((size_t)layer * c.pages + w.moves[2 * k]) * page_bytes;
        const size_t to = ((size_t)layer * c.pages + w.moves[2 * k + 1]) * page_bytes;
        copy_bytes16(pool + to, pool + from, (int)(page_bytes - b < (size_t)kCopyChunk ? page_bytes - b : (size_t)kCopyChunk));
    }
}

// ------------------------------------------------------------------------------------------
// launches
// ------------------------------------------------------------------------------------------
static cudaError_t sm_count(int* sms) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    return e == cudaSuccess ? cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) : e;
}

// a launch that (pdl 1) may begin while the one before it on the stream ends (its kernel waits for that one's results)
template <typename... KArgs, typename... Args>
static cudaError_t launch_after(void (*kern)(KArgs...), int grid, int threads, int pdl, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

cudaError_t launch_paged_resize(const PagedKv& c, const PagedWorkspace& w, int n, const int* seqs, const int* lens,
                                int add, int* pos, int pdl, cudaStream_t s, const PagedFrames* frames) {
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    CopyParts cp{};
    if (frames)
        for (cp.n = 0; cp.n < frames->n_parts; ++cp.n) cp.p[cp.n] = frames->parts[cp.n];
    paged_resize_kernel<<<1, kPT, 0, s>>>(c, w, n, seqs, lens, add, pos, frames ? frames->count : nullptr);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_after(paged_copy_kernel, sms, kCopyThreads, pdl, s, c, w, n, (const int*)nullptr, seqs, cp);
}

cudaError_t launch_paged_fork(const PagedKv& c, const PagedWorkspace& w, int n, const int* src, const int* dst,
                              const vc_session_part* parts, int n_parts, int* done, cudaStream_t s) {
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    CopyParts cp{};
    cp.n = n_parts;
    for (int i = 0; i < n_parts; ++i) cp.p[i] = parts[i];
    paged_fork_kernel<<<1, kPT, 0, s>>>(c, w, n, src, dst, done);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_after(paged_copy_kernel, 8 * sms, kCopyThreads, 1, s, c, w, n, src, dst, cp);
}

cudaError_t launch_paged_compact(const PagedKv& c, const PagedWorkspace& w, int* live, cudaStream_t s) {
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int chunks = (c.pages + kCompactChunk - 1) / kCompactChunk;
    paged_count_kernel<<<chunks, kCT, 0, s>>>(c, w);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_after(paged_list_kernel, chunks, kCT, 1, s, c, w, live)) != cudaSuccess) return e;
    return launch_after(paged_move_kernel, 8 * sms, kCopyThreads, 1, s, c, w);
}

}  // namespace vc
