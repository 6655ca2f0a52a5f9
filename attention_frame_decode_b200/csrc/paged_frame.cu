// paged_frame.cu -- windowed attention over the paged KV cache for single frames (one row per session).
//
// Bound: HBM.  A frame reads min(ctx, window + sinks) keys and values per session and KV head once, 4 Dh bytes
// each, and does 4 G Dh flops on them (G = q_heads / kv_heads query heads share them).
//
// The work of all sessions is one line of units (session, KV head, block of BK keys), cut into equal ranges, one
// for each warp of one CTA per SM: however ragged the sessions are, every SM reads the same amount.  A warp goes
// through its range without meeting another: it keeps a ring of TMA copies ahead of it (K and V blocks, swizzled
// rows, fetched page by page through the table) and the running maximum, sum and output of the softmax in registers.  The products
// run on warp-level matrix instructions with the keys (then the head dims) as the 16 rows and the query heads as
// the 8 columns, S^T = K Q^T and O^T = V^T P^T: up to 8 heads waste no row, and P^T is S^T's registers transposed.
// A (session, KV head) inside a range is written where it ends; one that ranges share leaves a record from each:
// the CTA joins its warps' records at the end, and where CTAs share it the last of them to arrive joins theirs, in
// order, so that results do not depend on timing.
// The weights go into the products as a 16-bit value and the 16-bit rest of it: the error of a weight is
// 2^-16 (bf16), and the products are not what this kernel waits for.  Of an infinite value that is seen they make NaN: results
// that are not finite are decided by the values themselves (paged_dev.cuh).
#include <algorithm>

#include "paged_dev.cuh"
#include "tc.cuh"

namespace vc {

static constexpr int kFMaxStages = 4;   // below eight (see look_up)
static constexpr int kFMaxBatch = 2048;
// Whole (session, KV head)s go to warps, and no join is needed, where that gives no warp more than this many units
// over an equal share: a join costs about as much as four units (2 us).  64 sessions, 40 heads over 8 of 128, whole and cut:
// behind 100 positions (4 units over the share) 13.7 and 19.2 us, 130 (6) 16.0 and 19.8, 200 (8) 20.2 and 21.7, 300 (11) 27.2
// and 25.4; one share or less a warp (16 sessions): 100 (6) 12.4 and 13.7, 200 (12) 17.8 and 16.8.
static constexpr int kWholeUnits = 4;

template <int DH>
struct FrameShape {
    static constexpr int WARPS = DH >= 256 ? 4 : 8, THREADS = 32 * WARPS;
    static constexpr int BK = DH >= 128 ? 16 : DH == 64 ? 32 : 64;    // keys per unit
    static constexpr int CS = DH + 4;                                  // floats per head in the joining buffer
    static constexpr int ROWB = DH >= 64 ? 128 : 64;                  // bytes per swizzled row
    static constexpr int PARTS = DH >= 64 ? DH / 64 : 1;              // column parts of a K or V block
    static constexpr int KBYTES = BK * DH * 2, STAGE = 2 * KBYTES;
    static constexpr int CH = DH / 8;                                  // 16-byte chunks per row
    // byte offset of chunk c of row r in a K or V block
    static VC_DEV uint32_t at(int r, int c) {
        if constexpr (DH >= 64)
            return (uint32_t)((c >> 3) * (BK * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
        else
            return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    }
};

struct FrameLayout {
    int stages;
    int off_comb, off_weights, off_sessions;   // after the rings
    size_t total;
};

template <int DH>
static FrameLayout frame_layout(int G, int batch, int grid) {
    using S = FrameShape<DH>;
    FrameLayout L{};
    const int comb = S::WARPS * ((G * (S::CS + 2) + 3) & ~3) * 4, weights = grid * (2 * G + 1) * 4, sessions = (batch + 1) * 16;
    const int rest = comb + weights + sessions + 1024 + 64;
    L.stages = (227 * 1024 - rest - 512) / (S::WARPS * S::STAGE);
    if (L.stages > kFMaxStages) L.stages = kFMaxStages;
    L.off_comb = S::WARPS * L.stages * S::STAGE;
    L.off_weights = L.off_comb + comb;
    L.off_sessions = (L.off_weights + weights + 15) / 16 * 16;
    L.total = (size_t)L.off_sessions + sessions + 1024;
    return L;
}

// a session of the line: its first unit, blocks per KV head, index in the cache, the row's position
struct LineSession {
    int first, blocks, s, p;
};

VC_DEV uint32_t transpose8x8(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

// NH: groups of 8 query heads (1 for up to 8 heads to a KV head, else 2)
template <int DH, bool F16, int NH>
__global__ void __launch_bounds__(FrameShape<DH>::THREADS, 1)
    paged_frame_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const PagedAttnArgs a, const FrameLayout L) {
    using S = FrameShape<DH>;
    constexpr int BK = S::BK, KT = BK / 16, MT = DH / 16, CS = S::CS, kWarps = S::WARPS, kThreads = S::THREADS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* comb = reinterpret_cast<float*>(smem + L.off_comb);        // records: [warps]{[G][CS], [G][2]}
    float* wts = reinterpret_cast<float*>(smem + L.off_weights);      // [CTAs][G][2], then [CTAs] records
    LineSession* line = reinterpret_cast<LineSession*>(smem + L.off_sessions);   // [batch + 1]
    __shared__ uint64_t full[kWarps][kFMaxStages];
    __shared__ uint32_t stage_mapped[kWarps][kFMaxStages];
    __shared__ int warp_total[kWarps], warp_most[kWarps];
    __shared__ int4 open_seg[2];   // what the CTA shares at its range's start and end: first unit, end, row, KV head
    __shared__ int open_last[2];   // whether this CTA arrived last

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
    const int G = a.c.Hq / a.c.Hk, Hk = a.c.Hk;
    pdl_trigger();
    if (lane == 0) {
        for (int s = 0; s < L.stages; ++s) mbar_init(&full[warp][s], 1);
        fence_mbar_init();
    }
    if (tid == 0) {
        tma_prefetch_map(&tmK);
        tma_prefetch_map(&tmV);
    }
    if (tid < 2) open_seg[tid] = make_int4(0, 0, 0, 0);
    pdl_wait();

    // the line's sessions (every CTA lays out the same line)
    int units = 0, heads_total = 0, most = 0;   // (session, KV head)s that have units, the most units of one
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        const int b = b0 + tid;
        LineSession me{0, 0, 0, 0};
        if (b < a.batch) {
            AttnSession o;
            if (attn_session(a, b, o)) {
                me.s = o.s;
                me.p = o.p0;
                me.blocks = key_blocks<BK>(a.c.window, a.c.sinks, o.p0, o.p0).total;
            }
        }
        int incl = me.blocks * Hk;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        const int top = __reduce_max_sync(0xffffffffu, me.blocks);
        if (lane == 31) {
            warp_total[warp] = incl;
            warp_most[warp] = top;
        }
        __syncthreads();
        int before = units;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += warp_total[w];
            units += warp_total[w];
            most = max(most, warp_most[w]);
        }
        me.first = before + incl - me.blocks * Hk;
        if (b < a.batch) line[b] = me;
        heads_total += Hk * __syncthreads_count(me.blocks > 0);
    }
    if (tid == 0) line[a.batch] = LineSession{units, 0, 0, 0};
    __syncthreads();
    if (units == 0) return;

    const int all_warps = (int)gridDim.x * kWarps;
    const bool whole_heads = most - (heads_total <= all_warps ? units / all_warps : 0) <= kWholeUnits;
    // ranges of a unit at least (short lines: fewer records to join), the first `more` one unit longer
    const int ctas = whole_heads ? (int)gridDim.x : max(1, min((int)gridDim.x, units / kWarps));
    if ((int)blockIdx.x >= ctas) return;
    const int ranges = ctas * kWarps, share = units / ranges, more = units - share * ranges;
    auto range_start = [&](int c) { return c * share + min(c, more); };
    auto owner = [&](int x) {
        const int cut = more * (share + 1);
        return x < cut ? x / (share + 1) : more + (x - cut) / max(share, 1);
    };
    auto session_at = [&](int x) {   // the last session that starts at or before unit x
        int lo = 0, hi = a.batch - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (line[mid].first <= x) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    const int range0 = whole_heads ? 0 : (int)blockIdx.x * kWarps;   // the CTA's first range
    const int range = whole_heads ? warp * (int)gridDim.x + (int)blockIdx.x : range0 + warp;
    int c0 = range_start(range), c1 = range_start(range + 1);
    if (whole_heads) {   // the (session, KV head)s whose first unit lies in the range
        auto next_head = [&](int x) {
            if (x >= units) return units;
            const LineSession me = line[session_at(x)];
            return me.first + (x - me.first + me.blocks - 1) / me.blocks * me.blocks;
        };
        c0 = next_head(c0);
        c1 = next_head(c1);
    }

    // a place on the line: a unit is block `blk` of session b's KV head j
    struct Place {
        int b, j, blk;
    };
    auto forward = [&](Place& u, int by) {   // `by` units on
        u.blk += by;
        int n = line[u.b].blocks;
        while (u.blk >= n) {
            u.blk -= n;
            if (++u.j == Hk) {
                u.j = 0;
                do ++u.b;
                while (u.b < a.batch && line[u.b].blocks == 0);
                if (u.b >= a.batch) return;   // behind the line's end
                n = line[u.b].blocks;
            }
        }
    };
    Place here{0, 0, 0};   // the range's first unit
    if (c0 < c1) {
        const int b = session_at(c0), rel = c0 - line[b].first, n = line[b].blocks;
        here = Place{b, rel / n, rel % n};
    }

    // ---- this warp's copies: unit c0 + i is copy i, in ring slot i % stages ----
    uint8_t* ring = smem + (size_t)warp * L.stages * S::STAGE;
    const int box_rows = min(a.c.page, BK), boxes = BK / box_rows, batch = 32 / boxes;
    const int copies = max(c1 - c0, 0);
    int copy = 0, copy_slot = 0, looked = 0;
    Place look = here;
    // looks up the pages of the next `batch` copies: lane batch i + q gets the table entry of copy i's q-th box
    // (-1: none) and its row within the page; two batches are held, so that no copy waits for its entry
    struct Look {
        int entry, row;
    };
    auto look_up = [&]() {
        Look o{-1, 0};
        const int i = lane / boxes;
        if (looked + i < copies) {
            Place u = look;
            if (i) forward(u, i);
            const LineSession me = line[u.b];
            const KeyBlocks kb = key_blocks<BK>(a.c.window, a.c.sinks, me.p, me.p);
            const int t = kb.block(u.blk) * BK + (lane & (boxes - 1)) * box_rows;
            o.row = u.j * a.c.page + (t & (a.c.page - 1));
            if (t <= me.p) o.entry = a.c.table[(size_t)me.s * a.c.columns + (t >> a.c.page_shift)];
        }
        looked += batch;
        if (looked < copies) forward(look, batch);
        return o;
    };
    Look now = look_up(), next{-1, 0};
    auto issue = [&]() {   // starts the next copy
        if (copy >= copies) return;
        const int from = copy % batch * boxes + (lane & (boxes - 1));
        const int entry = __shfl_sync(0xffffffffu, now.entry, from), row = __shfl_sync(0xffffffffu, now.row, from);
        const bool there = lane < boxes && (unsigned)entry < (unsigned)a.c.pages;
        const unsigned mapped = __ballot_sync(0xffffffffu, there);
        uint64_t* bar = &full[warp][copy_slot];
        if (lane == 0) {
            stage_mapped[warp][copy_slot] = mapped;
            mbar_arrive_expect_tx(bar, (uint32_t)(__popc(mapped) * box_rows * DH * 4));
        }
        __syncwarp();
        if (there) {
            const int pool_row = entry * Hk * a.c.page + row;
            uint8_t* to = ring + copy_slot * S::STAGE + lane * box_rows * S::ROWB;
#pragma unroll
            for (int part = 0; part < S::PARTS; ++part) {
                tma_load_2d(to + part * (BK * 128), &tmK, part * 64, pool_row, bar);
                tma_load_2d(to + S::KBYTES + part * (BK * 128), &tmV, part * 64, pool_row, bar);
            }
        }
        copy_slot = copy_slot + 1 == L.stages ? 0 : copy_slot + 1;
        if (++copy % batch == 0) {
            now = next;
            next = look_up();
        }
    };
#pragma unroll 1
    for (int s = 0; s < L.stages; ++s) issue();
    next = look_up();   // (a batch is at least eight copies: the first stages come from the first)

    auto out_at = [&](int row, int j, int r, int d) { return a.out + (size_t)row * a.out_ld + (size_t)(j * G + r) * DH + d; };
    auto rec_a = [&](int w) { return comb + (size_t)w * ((G * (CS + 2) + 3) & ~3); };   // 16-byte aligned
    auto rec_b = [&](int w) { return reinterpret_cast<float*>(smem + (size_t)w * L.stages * S::STAGE); };

    // ---- units ----
    int slot = 0, phase = 0, used = 0;
    bool alive = true;   // false after a copy that never came: nothing more is computed, the barriers are kept
    const int mi = lane >> 3, lr = lane & 7;
    // what two warps of the CTA share: (first unit, end, row, KV head) of the range's first and last segment
    int4 seg_first = make_int4(0, 0, 0, 0), seg_last = seg_first;
    for (int x_seg = c0; x_seg < c1;) {
        const Place at0 = here;   // of unit x_seg
        const int b = at0.b;
        const LineSession me = line[b];
        const int s0 = me.first + at0.j * me.blocks, s1 = s0 + me.blocks, end = min(s1, c1);
        const KeyBlocks kb = key_blocks<BK>(a.c.window, a.c.sinks, me.p, me.p);
        const int row = b;
        uint32_t qb[MT][NH][2];   // Q^T: dims 16 ks + 2 tq .. of heads 8 h + g
        {
            const uint16_t* q0 = a.q + (size_t)row * a.q_ld + (size_t)(at0.j * G) * DH + 2 * tq;
#pragma unroll
            for (int ks = 0; ks < MT; ++ks)
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const uint16_t* qr = q0 + (size_t)(8 * h + g) * DH + ks * 16;
                    qb[ks][h][0] = 8 * h + g < G ? *reinterpret_cast<const uint32_t*>(qr) : 0u;
                    qb[ks][h][1] = 8 * h + g < G ? *reinterpret_cast<const uint32_t*>(qr + 8) : 0u;
                }
        }
        // the new row's key and value and its page, for the warp that has the segment's last block
        uint4 new_k = make_uint4(0u, 0u, 0u, 0u), new_v = new_k;
        int new_page = -1;
        if (a.kn && s1 <= c1 && lane < S::CH) {
            new_k = *reinterpret_cast<const uint4*>(a.kn + (size_t)row * a.k_ld + at0.j * DH + lane * 8);
            new_v = *reinterpret_cast<const uint4*>(a.vn + (size_t)row * a.v_ld + at0.j * DH + lane * 8);
            new_page = page_of(a.c, me.s, me.p >> a.c.page_shift);
        }
        float acc[MT][NH][4];   // O^T: dims 16 mt + g (+ 8) of heads 8 h + 2 tq (+ 1)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < NH; ++h) acc[mt][h][0] = acc[mt][h][1] = acc[mt][h][2] = acc[mt][h][3] = 0.0f;
        float m[NH][2], l[NH][2];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            m[h][0] = m[h][1] = -INFINITY;
            l[h][0] = l[h][1] = 0.0f;
        }

        for (int x = x_seg; x < end; ++x) {
            ++used;
            if (alive) {
                alive = __all_sync(0xffffffffu, mbar_wait(&full[warp][slot], phase, a.c.status));
                if (!alive)   // the copies behind it are given another bounded while before anyone leaves
                    for (int k = used, sl = slot, ph = phase; k < copy; ++k) {
                        if (++sl == L.stages) sl = 0, ph ^= 1;
                        mbar_wait(&full[warp][sl], ph, nullptr);
                    }
            }
            if (alive) {
                uint8_t* Ks = ring + slot * S::STAGE;
                uint8_t* Vs = Ks + S::KBYTES;
                const unsigned mapped = stage_mapped[warp][slot];
                const int t0 = kb.block(x - s0) * BK, p = me.p;
                auto seen = [&](int r) {
                    const int t = t0 + r;
                    return ((mapped >> (r / box_rows)) & 1u) && t <= p &&
                           (a.c.window == 0 || t < a.c.sinks || t > p - a.c.window);
                };
                const bool whole = mapped == (1u << boxes) - 1u && t0 + BK - 1 <= p &&
                                   (a.c.window == 0 || t0 > p - a.c.window || t0 + BK - 1 < a.c.sinks);
                const bool newest = a.kn && t0 <= p && p < t0 + BK;
                if (!whole || newest) {
                    // values that nothing sees must not reach the products, whatever they are
                    for (int i = lane; i < BK * S::CH; i += 32)
                        if (!seen(i / S::CH))
                            *reinterpret_cast<uint4*>(Vs + S::at(i / S::CH, i % S::CH)) = make_uint4(0u, 0u, 0u, 0u);
                    __syncwarp();
                    if (newest && new_page >= 0) {   // the new row, into the block
                        *reinterpret_cast<uint4*>(Ks + S::at(p - t0, lane)) = new_k;
                        *reinterpret_cast<uint4*>(Vs + S::at(p - t0, lane)) = new_v;
                    }
                    __syncwarp();
                }
                float sc[KT][NH][4];   // S^T: keys 16 kt + g (+ 8), heads 8 h + 2 tq (+ 1)
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int h = 0; h < NH; ++h) sc[kt][h][0] = sc[kt][h][1] = sc[kt][h][2] = sc[kt][h][3] = 0.0f;
#pragma unroll
                for (int ks = 0; ks < MT; ++ks)
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        uint32_t kf[4];
                        ldsm4(kf, Ks + S::at(16 * kt + 8 * (mi & 1) + lr, 2 * ks + (mi >> 1)));
#pragma unroll
                        for (int h = 0; h < NH; ++h) mma16<F16>(sc[kt][h], kf, qb[ks][h][0], qb[ks][h][1]);
                    }
                bool hide[KT][2];   // keys that are not seen
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int u = 0; u < 2; ++u) hide[kt][u] = !whole && !seen(16 * kt + g + 8 * u);
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    float base[2], corr[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = m[h][e];
#pragma unroll
                        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                float& z = sc[kt][h][2 * u + e];
                                z = hide[kt][u] ? -INFINITY : z * a.scale_log2;
                                mx = fmaxf(mx, z);
                            }
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        base[e] = mx == -INFINITY ? 0.0f : mx;
                        corr[e] = exp2_approx(m[h][e] - base[e]);
                        m[h][e] = mx;
                        l[h][e] *= corr[e];
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        acc[mt][h][0] *= corr[0]; acc[mt][h][1] *= corr[1];
                        acc[mt][h][2] *= corr[0]; acc[mt][h][3] *= corr[1];
                    }
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            sc[kt][h][u] = exp2_approx(sc[kt][h][u] - base[u & 1]);
                            l[h][u & 1] += sc[kt][h][u];
                        }
                }
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    uint32_t hi[NH][2], lo[NH][2];   // P^T: keys 2 tq (+ 8 u), head g
#pragma unroll
                    for (int h = 0; h < NH; ++h)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float w0 = sc[kt][h][2 * u], w1 = sc[kt][h][2 * u + 1];
                            const uint32_t v = pack16<F16>(w0, w1);
                            hi[h][u] = transpose8x8(v);
                            lo[h][u] = transpose8x8(pack16<F16>(w0 - unpack16<F16>((uint16_t)v), w1 - unpack16<F16>((uint16_t)(v >> 16))));
                        }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t vf[4];
                        ldsm4_t(vf, Vs + S::at(16 * kt + 8 * (mi >> 1) + lr, 2 * mt + (mi & 1)));
#pragma unroll
                        for (int h = 0; h < NH; ++h) {
                            mma16<F16>(acc[mt][h], vf, hi[h][0], hi[h][1]);
                            mma16<F16>(acc[mt][h], vf, lo[h][0], lo[h][1]);
                        }
                    }
                }
                if (!whole || newest) fence_proxy_async();   // stores to the slot come before the next copy into it
                __syncwarp();
                issue();
                if (newest && new_page >= 0) {   // and to its page
                    const size_t to = (((size_t)new_page * Hk + at0.j) * a.c.page + (p & (a.c.page - 1))) * DH + lane * 8;
                    *reinterpret_cast<uint4*>(a.c.k + to) = new_k;
                    *reinterpret_cast<uint4*>(a.c.v + to) = new_v;
                }
            }
            if (++slot == L.stages) {
                slot = 0;
                phase ^= 1;
            }
        }
        // ---- the end of the (session, KV head), or of the range ----
        const bool ends_here = s0 >= c0 && s1 <= c1;
        float* rec = x_seg == c0 ? rec_a(warp) : rec_b(warp);   // the ring is free where the range ends
        unsigned odd = 0;   // heads of which a result is not finite and the weights' sum is a number
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[h][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int r = 8 * h + 2 * tq + e;
                if (r >= G) continue;
                if (ends_here) {
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                    uint16_t* to = out_at(row, at0.j, r, g);
                    float x = 0.0f;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) x += acc[mt][h][e] * 0.0f + acc[mt][h][2 + e] * 0.0f;
                    if (x != 0.0f && sum == sum) odd |= 1u << r;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const uint32_t v = pack_out<F16>(a.widen, acc[mt][h][e] * inv, acc[mt][h][2 + e] * inv);
                        to[16 * mt] = (uint16_t)v;
                        to[16 * mt + 8] = (uint16_t)(v >> 16);
                    }
                } else {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        rec[r * CS + 16 * mt + g] = acc[mt][h][e];
                        rec[r * CS + 16 * mt + g + 8] = acc[mt][h][2 + e];
                    }
                    if (g == 0) *reinterpret_cast<float2*>(rec + G * CS + 2 * r) = make_float2(m[h][e], sum);
                }
            }
        if (__any_sync(0xffffffffu, odd != 0)) {
            odd = __reduce_or_sync(0xffffffffu, odd);
            __threadfence_block();
            __syncwarp();   // the outputs, and the new row in its page
            const SeenValues<DH> values = seen_values<DH>(a.c, me.s, at0.j, me.p);
#pragma unroll 1
            for (int d = 4 * lane; d < DH; d += 128) {
                const float4 z = odd_values_call<DH, F16>(values, d);
#pragma unroll 1
                for (int r = 0; r < G; ++r) {
                    if (!((odd >> r) & 1u)) continue;
                    uint16_t* to = out_at(row, at0.j, r, d);
                    if (z.x != 0.0f) to[0] = (uint16_t)pack_out<F16>(a.widen, z.x, 0.0f);
                    if (z.y != 0.0f) to[1] = (uint16_t)pack_out<F16>(a.widen, z.y, 0.0f);
                    if (z.z != 0.0f) to[2] = (uint16_t)pack_out<F16>(a.widen, z.z, 0.0f);
                    if (z.w != 0.0f) to[3] = (uint16_t)pack_out<F16>(a.widen, z.w, 0.0f);
                }
            }
        }
        if (!ends_here) {
            seg_last = make_int4(s0, s1, row, at0.j);
            if (x_seg == c0) seg_first = seg_last;
        }
        if (end < c1) forward(here, end - x_seg);
        x_seg = end;
    }
    if (whole_heads) return;

    // ---- the CTA's warps: each joins what begins with it (warp 0: also what began before the CTA) ----
    __syncthreads();
    const int rec_floats = (G * (DH + 2) + 3) & ~3;   // 16-byte aligned records
    auto decide = [&](float (&v)[4], float sum, const int4& seg, int d) {   // results of a segment's row (times its sum or not)
        if (odd_results(v) && sum == sum)
            decide_odd(v, odd_values_call<DH, F16>(seen_values<DH>(a.c, line[seg.z].s, seg.w, line[seg.z].p), d));
    };
    const int C0 = range_start(range0), C1 = range_start(range0 + kWarps);
    auto join_warps = [&](const int4& seg) {
        const int s0 = seg.x, s1 = seg.y, last = owner(min(s1, C1) - 1) - range0;
        const bool shared = s0 < C0 || s1 > C1;
        const int which = s0 <= C0 ? 0 : 1;
        float* rec = a.partial + (size_t)(2 * blockIdx.x + which) * rec_floats;
        const float* from[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w)   // a warp's first segment is in its first record
            from[w] = w < warp || w > last ? nullptr : s0 <= range_start(range0 + w) ? rec_a(w) : rec_b(w);
        for (int i = lane; i < G * (DH / 4); i += 32) {
            const int r = i / (DH / 4), d = 4 * (i % (DH / 4));
            // a part without a key that is seen has maximum -inf, sum 0 and zeros: its factor is 0
            float top = -INFINITY, f[kWarps], sum = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                f[w] = from[w] ? from[w][G * CS + 2 * r] : -INFINITY;
                top = fmaxf(top, f[w]);
            }
            const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (!from[w]) continue;
                f[w] = exp2_approx(f[w] - base);
                const float4 y = *reinterpret_cast<const float4*>(from[w] + r * CS + d);
                sum = fmaf(from[w][G * CS + 2 * r + 1], f[w], sum);
                v[0] = fmaf(y.x, f[w], v[0]); v[1] = fmaf(y.y, f[w], v[1]);
                v[2] = fmaf(y.z, f[w], v[2]); v[3] = fmaf(y.w, f[w], v[3]);
            }
            if (!shared) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                decide(v, sum, seg, d);
                *reinterpret_cast<uint2*>(out_at(seg.z, seg.w, r, d)) =
                    make_uint2(pack_out<F16>(a.widen, v[0] * inv, v[1] * inv), pack_out<F16>(a.widen, v[2] * inv, v[3] * inv));
            } else {
                __stcg(reinterpret_cast<float4*>(rec + r * DH + d), make_float4(v[0], v[1], v[2], v[3]));
                if (d == 0) __stcg(reinterpret_cast<float2*>(rec + G * DH + 2 * r), make_float2(top, sum));
            }
        }
        if (shared && lane == 0) open_seg[which] = seg;
    };
    if (warp == 0 && seg_first.y > seg_first.x) join_warps(seg_first);
    if (seg_last.y > c1 && seg_last.x >= c0 && !(warp == 0 && seg_last.x <= c0)) join_warps(seg_last);

    // ---- the CTAs ----
    __syncthreads();
    if (tid < 2) {
        const int4 seg = open_seg[tid];
        int is_last = 0;
        if (seg.y > seg.x) {
            __threadfence();   // the CTA's records, ordered by the barrier, before its arrival
            const int f = owner(seg.x) / kWarps, n = owner(seg.y - 1) / kWarps - f + 1;
            is_last = atomicAdd(a.merge + f, 1) == n - 1;
            if (is_last) a.merge[f] = 0;
            __threadfence();
        }
        open_last[tid] = is_last;
    }
    __syncthreads();
    // up to twelve contributors: a thread takes four columns of a row with everything that it needs in flight at once
    // (the maxima and sums are the same addresses for the row's threads)
    // Twelve, since room for more (registers) costs every join: one session, 40 heads over 8 of 128, under a window of 1024
    // with 64 sinks (10 contributors to a KV head) 13.5 us, 14.8 with room for 20, 15.7 in the form below; without a window
    // behind 2000 positions (17) 16.2 (the form below), 15.3 with room for 20; 16 sessions behind 4096 (2 or 3) 56.3, 57.6,
    // 58.5.
    constexpr int kFew = 12;
    const int pieces = G * (DH / 4);
    auto record_of = [&](const int4& seg, int cta) { return (2 * cta + (seg.x <= range_start(cta * kWarps) ? 0 : 1)) * rec_floats; };
    for (int i = tid; i < 2 * pieces; i += kThreads) {
        const int which = i >= pieces, r = i % pieces / (DH / 4), d = 4 * (i % (DH / 4));
        const int4 seg = open_seg[which];
        if (!open_last[which]) continue;
        const int f = owner(seg.x) / kWarps, n = owner(seg.y - 1) / kWarps - f + 1;
        if (n > kFew) continue;
        float2 w[kFew];
        float4 y[kFew];
#pragma unroll
        for (int k = 0; k < kFew; ++k) {
            const float* rec = a.partial + (k < n ? record_of(seg, f + k) : 0);
            w[k] = k < n ? __ldcg(reinterpret_cast<const float2*>(rec + G * DH + 2 * r)) : make_float2(-INFINITY, 0.0f);
            y[k] = k < n ? __ldcg(reinterpret_cast<const float4*>(rec + r * DH + d)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        float top = -INFINITY, sum = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < kFew; ++k) top = fmaxf(top, w[k].x);
        if (top == -INFINITY) top = 0.0f;
#pragma unroll
        for (int k = 0; k < kFew; ++k) {
            const float x = exp2_approx(w[k].x - top);
            sum = fmaf(w[k].y, x, sum);
            v[0] = fmaf(y[k].x, x, v[0]); v[1] = fmaf(y[k].y, x, v[1]);
            v[2] = fmaf(y[k].z, x, v[2]); v[3] = fmaf(y[k].w, x, v[3]);
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        decide(v, sum, seg, d);
        *reinterpret_cast<uint2*>(out_at(seg.z, seg.w, r, d)) =
            make_uint2(pack_out<F16>(a.widen, v[0] * inv, v[1] * inv), pack_out<F16>(a.widen, v[2] * inv, v[3] * inv));
    }
    for (int which = 0; which < 2; ++which) {
        if (!open_last[which]) continue;
        const int4 seg = open_seg[which];
        const int f = owner(seg.x) / kWarps, n = owner(seg.y - 1) / kWarps - f + 1;
        if (n <= kFew) continue;
        // wts[k][r]: the k-th contributor's (maximum, sum), then its factor; its record is that of its range's start
        // if the segment began there or before
        int* rec_at = reinterpret_cast<int*>(wts + 2 * n * G);
        for (int k = tid; k < n; k += kThreads)
            rec_at[k] = record_of(seg, f + k);
        __syncthreads();
        for (int i = tid; i < n * G; i += kThreads)
            reinterpret_cast<float2*>(wts)[i] =
                __ldcg(reinterpret_cast<const float2*>(a.partial + rec_at[i / G] + G * DH + 2 * (i % G)));
        __syncthreads();
        for (int r = warp; r < G; r += kWarps) {
            float top = -INFINITY, sum = 0.0f;
            for (int k = lane; k < n; k += 32) top = fmaxf(top, wts[2 * (k * G + r)]);
            top = warp_max(top);
            if (top == -INFINITY) top = 0.0f;
            for (int k = lane; k < n; k += 32) {
                float* w = wts + 2 * (k * G + r);
                const float f2 = exp2_approx(w[0] - top);
                sum = fmaf(w[1], f2, sum);
                w[0] = f2;
            }
            sum = warp_sum(sum);
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            for (int k = lane; k < n; k += 32) wts[2 * (k * G + r)] *= inv;
        }
        __syncthreads();
        for (int i = tid; i < G * (DH / 4); i += kThreads) {
            const int r = i / (DH / 4), d = 4 * (i % (DH / 4));
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
            for (int k = 0; k < n; ++k) {
                const float4 y = __ldcg(reinterpret_cast<const float4*>(a.partial + rec_at[k] + r * DH + d));
                const float w = wts[2 * (k * G + r)];
                v[0] = fmaf(y.x, w, v[0]); v[1] = fmaf(y.y, w, v[1]);
                v[2] = fmaf(y.z, w, v[2]); v[3] = fmaf(y.w, w, v[3]);
            }
            decide(v, wts[2 * r], seg, d);
            *reinterpret_cast<uint2*>(out_at(seg.z, seg.w, r, d)) =
                make_uint2(pack_out<F16>(a.widen, v[0], v[1]), pack_out<F16>(a.widen, v[2], v[3]));
        }
        __syncthreads();   // the factors' room is used again
    }
}

template <int DH, bool F16>
static cudaError_t launch_frames_t(const PagedAttnArgs& a, cudaStream_t s) {
    using S = FrameShape<DH>;
    const int grid = a.num_sms;
    const FrameLayout L = frame_layout<DH>(a.c.Hq / a.c.Hk, a.batch, grid);
    if (L.stages < 2) return cudaErrorNotSupported;
    CUtensorMap mk, mv;
    const int rows = a.c.pages * a.c.Hk * a.c.page, box = a.c.page < S::BK ? a.c.page : S::BK;
    const CUtensorMapSwizzle swz = DH >= 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    if (!tma_map_2d(&mk, a.c.k, rows, DH, DH, DH < 64 ? DH : 64, box, F16, swz) ||
        !tma_map_2d(&mv, a.c.v, rows, DH, DH, DH < 64 ? DH : 64, box, F16, swz))
        return cudaErrorInvalidValue;
    auto kern = a.c.Hq / a.c.Hk <= 8 ? paged_frame_kernel<DH, F16, 1> : paged_frame_kernel<DH, F16, 2>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L.total);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(S::THREADS);
    cfg.dynamicSmemBytes = L.total;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = a.pdl;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, mk, mv, a, L);
}

cudaError_t launch_paged_frames(const PagedAttnArgs& a, cudaStream_t s) {
    // a line of units that 32 bits count, in blocks of at least 16 keys; up to 16 query heads to a KV head (the rows
    // of one matrix instruction); sessions that the line's table in shared memory holds
    long long reach = (long long)a.c.columns * a.c.page;
    if (a.c.window > 0) reach = std::min(reach, (long long)a.c.window + a.c.sinks);
    const long long most = reach / 16 + 4;
    if (a.c.Hq / a.c.Hk > 16 || a.batch > kFMaxBatch || most * a.c.Hk * a.batch > INT32_MAX) return cudaErrorNotSupported;
    switch (a.c.Dh) {
        case 32: return a.f16 ? launch_frames_t<32, true>(a, s) : launch_frames_t<32, false>(a, s);
        case 64: return a.f16 ? launch_frames_t<64, true>(a, s) : launch_frames_t<64, false>(a, s);
        case 128: return a.f16 ? launch_frames_t<128, true>(a, s) : launch_frames_t<128, false>(a, s);
        case 256: return a.f16 ? launch_frames_t<256, true>(a, s) : launch_frames_t<256, false>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace vc
