// paged_prompt.cu -- windowed attention over the paged KV cache for prompts, on tcgen05 tensor cores.
//
// The packed rows of a session and KV head (paged_attn.cu) are cut into tiles of 256 (head dim 128) or 512 rows (head
// dim 64): two or four MMA tiles of 128 rows.  One CTA per SM takes tiles in turn and walks the blocks of 128 or 64
// keys that a tile's rows can see.  Per block and MMA tile i:
//     S_i = Q_i K^T (tcgen05.mma into tensor memory, fp32)
//     P_i = exp2(scale S_i - m_i), 64 scores a thread, written back to tensor memory as the 16-bit A operand
//     O_i += P_i V (tcgen05.mma, A from tensor memory)
// The MMA tiles alternate: while the threads of one form its weights, the tensor core works on the others' products.
// m_i moves only where a row's highest score grew by more than 8 (a factor of 2^8), and what is checked on the way is
// the sum of a thread's 64 weights: at most 2^14, no weight is above it (the 16-bit types hold that; fp32 sums lose
// nothing by the common factor).  So O_i is rarely read back to be rescaled, a block's scores are passed over once, and
// no maximum is taken: at head dim 64, where issue slots and exponentials are what is short, that was worth 9%.
// Bound, per block of 128 keys x 256 rows (or 64 x 512) and SM: 2048 cycles of exponentials (8 a warp and register) and
// 2016 (head dim 128: M = N = 128, 63 each) or 1256 of products.  What it takes is the chain of one tile -- scores on
// their way 600 to 1300, weights 1100 alone, their way back 200 -- against the other tiles' chains: about 3400 cycles
// at head dim 128, whose tensor memory has no room for a third tile, and 2800 at head dim 64 with four tiles (with two
// tiles of 128 keys and two threads a row 3700: 219 us where four tiles take 198).
// Measured on a B200: 8192 rows of 40 heads over 8 of 128, window 4096, 64 sinks: 490 us at 1965 MHz, 1060 TFLOP/s of what
// the rows see, and 554 us, 941 TFLOP/s, in a loop of seconds (1725 MHz under the power cap); 12 blocks of 1 to 900 rows,
// 32 heads over 8 of 64, window 2048: 150 us with the longest tiles first (splitting the
// last round's key blocks gave back in records and joins what it evened out, and cost the other launch 2%).  A polynomial
// on the FMA units for every fourth or eighth exponential: 4 to 9% slower (issue slots).
// Warps: 0 copies K and V page by page (TMA, 128-byte swizzle) into a ring; 1 issues the MMAs; 2 hands out pieces and
// brings the rows of Q; 3 cleans the values of edge blocks; 4-19 are the rows.
#include "paged_dev.cuh"
#include "tc.cuh"

namespace vc {

static constexpr int kPThreads = 640;

template <int DH>
struct PromptShape {
    static constexpr int TILES = DH == 128 ? 2 : 4;           // MMA tiles of 128 rows
    static constexpr int KEYS = DH == 128 ? 128 : 64;         // keys of a block
    static constexpr int SHARES = KEYS / 64;                  // threads of a row, 64 scores of a block each
    static constexpr int ROWS = TILES * 128;
    static constexpr int HALVES = DH / 64;                    // 64-wide column parts
    static constexpr int TILE = KEYS * DH * 2;                // bytes of a K or V block
    static constexpr int QBYTES = ROWS * DH * 2;              // bytes of the rows of Q, [halves][rows][128 B]
    static constexpr int STAGES = DH == 128 ? 4 : 16;         // K and V blocks in turn (a power of two)
    static constexpr int BYTES = QBYTES + STAGES * TILE + 1024;
    static constexpr uint32_t ALL = (1u << (KEYS / 16)) - 1;  // every 16 keys of a block have a page
    // tensor memory columns: S of each tile, O of each tile.  P lies over S, each thread's weights over the scores that
    // they came from (the MMAs of one shape run in order, so S of the next block is written after P of this one is read)
    static constexpr uint32_t S0 = 0, O0 = TILES * KEYS;
    static_assert(TILES * (KEYS + DH) == 512 && TILES * 4 * SHARES == 16, "tensor memory, warps");
};

// a warpgroup's registers per thread, all four warps
template <bool MORE, int N>
VC_DEV void set_registers() {
    if constexpr (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// one lane of a converged warp.  What that lane alone does needs no proof that its operands are the same in all
// lanes: the products' descriptors go to uniform registers without a loop over the lanes.
VC_DEV bool elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
}
// D (tensor memory) (+)= A B^T, A from tensor memory
VC_DEV void tc_mma_ta(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 16 32-bit values of each lane to 16 consecutive columns
VC_DEV void tc_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
VC_DEV void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// maximum of three; NaN if one is
VC_DEV float max3(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// two fp32 operations in one instruction
VC_DEV float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
VC_DEV float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// the two warps (64 threads) of a row: whether any of their threads has p; a barrier
VC_DEV bool any_of_pair(int id, bool p) {
    uint32_t any;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.or.pred q, %1, 64, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(any)
        : "r"(id), "r"((uint32_t)p)
        : "memory");
    return any != 0;
}
VC_DEV void sync_pair(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }

// one of the steps of a 4 x 4 transpose over lanes: y of the lanes without the bit for x of those with it
VC_DEV void swap_lanes(uint4& x, uint4& y, int bit, bool has) {
    uint4 t = has ? x : y;
    t.x = __shfl_xor_sync(0xffffffffu, t.x, bit);
    t.y = __shfl_xor_sync(0xffffffffu, t.y, bit);
    t.z = __shfl_xor_sync(0xffffffffu, t.z, bit);
    t.w = __shfl_xor_sync(0xffffffffu, t.w, bit);
    if (has) x = t;
    else y = t;
}

VC_DEV void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// the low n bits (all for n >= 32, none for n <= 0)
VC_DEV uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// what a thread knows of its row
struct PromptRow {
    int p, window, sinks;
    // bit c: whether key t0 + c is seen (c < 32); groups: bit u, whether the 16 keys from t0 + 16 u on have a page
    VC_DEV uint32_t seen(int t0, uint32_t groups) const {
        uint32_t v = low_bits(p - t0 + 1);
        if (window > 0) v &= ~low_bits(p - window + 1 - t0) | low_bits(sinks - t0);
        return v & (((groups & 1u) ? 0xffffu : 0u) | ((groups & 2u) ? 0xffff0000u : 0u));
    }
};

struct PromptMaps {
    CUtensorMap q, k, v;
};

// one piece of work: a tile of a session and KV head, or a split of its key blocks
struct PromptWork {
    KeyBlocks kb;            // the tile's key blocks; this piece's are b0 .. b0 + nb - 1
    int b0, nb;
    int s, row0, n_rows;     // the session's index and first row; its packed rows
    int r0, r1, p0;          // the tile's packed rows r0 .. r1 - 1; the position of the session's first row
    int p_lo, p_hi, j;
    int splits, of, record;  // the launch's pieces of a tile; how many of them have blocks; this piece's record
};

// The launch's tiles, longest first, so that the CTAs end together: 12 blocks of 1 to 900 rows 147 us in this order, 181 in
// the sessions'.  Every CTA ranks them alike (the whole CTA calls; up to kSortTiles tiles and sessions).
static constexpr int kSortTiles = 512;
struct TileOrder {
    int first[kSortTiles + 1], key[kSortTiles], tile[kSortTiles];   // tile: session << 16 | tile within it, by rank
    int warp_sum[kPThreads / 32], count;
};
template <class S>
VC_DEV void order_tiles(const PagedAttnArgs& a, int most_tiles, TileOrder& o) {
    const int tid = threadIdx.x, lane = tid & 31, G = a.c.Hq / a.c.Hk, tile_rows = S::ROWS / G * G;
    const int mine = tid < a.batch ? (int)(((long long)session_rows(a, tid) * G + tile_rows - 1) / tile_rows) : 0;
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += u;
    }
    if (lane == 31) o.warp_sum[tid >> 5] = incl;
    __syncthreads();
    int before = incl - mine;
    for (int w = 0; w < tid >> 5; ++w) before += o.warp_sum[w];
    if (tid <= a.batch) o.first[tid] = before;   // (first[batch]: all of them)
    __syncthreads();
    const int count = min(o.first[a.batch], most_tiles);   // more only where cu_rows overlap (those sessions are refused)
    int key = 0, at = 0;
    if (tid < count) {
        int lo = 0, hi = a.batch - 1;   // the last session that starts at or before the tile
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (o.first[mid] <= tid) lo = mid;
            else hi = mid - 1;
        }
        const int tile = tid - o.first[lo], r0 = tile * tile_rows, r1 = min(r0 + tile_rows, session_rows(a, lo) * G), p0 = a.pos[lo];
        at = lo << 16 | tile;
        if (p0 >= 0 && p0 < 1 << 30)   // key blocks, and what one takes by the MMA tiles that have rows
            key = key_blocks<S::KEYS>(a.c.window, a.c.sinks, p0 + r0 / G, p0 + (r1 - 1) / G).total * ((r1 - r0 + 127) / 128 + 3);
        o.key[tid] = key;
    }
    __syncthreads();
    if (tid < count) {
        int rank = 0;
        for (int k = 0; k < count; ++k) rank += o.key[k] > key || (o.key[k] == key && k < tid);
        o.tile[rank] = at;
    }
    if (tid == 0) o.count = count;
    __syncthreads();
}

// piece `item` of the launch (a whole warp calls); nb is 0 where there is nothing to do, and n_rows too where not even
// an empty record is wanted, and -1 behind the last piece.  A tile holds whole tokens: tile_rows = (ROWS / G) G rows.
template <class S>
VC_DEV PromptWork prompt_work(const PagedAttnArgs& a, const TileOrder* order, int tiles, int splits, int item) {
    PromptWork w{};
    const int G = a.c.Hq / a.c.Hk, tile_rows = S::ROWS / G * G;
    if (item >= tiles * a.c.Hk * splits) {
        w.nb = -1;
        return w;
    }
    const int unit = item / splits, split = item % splits;
    w.record = item;
    w.splits = splits;
    w.j = unit % a.c.Hk;
    int session, tile;
    AttnSession o;
    if (order) {
        session = order->tile[unit / a.c.Hk] >> 16;
        tile = order->tile[unit / a.c.Hk] & 0xffff;
    } else if (!find_tile(a, G, tile_rows, tiles - 1 - unit / a.c.Hk, session, tile)) {   // a session's last rows first
        return w;
    }
    if (!attn_session(a, session, o)) return w;
    w.s = o.s;
    w.row0 = o.row0;
    w.n_rows = o.n * G;
    w.r0 = tile * tile_rows;
    w.p0 = o.p0;
    w.p_lo = o.p0 + w.r0 / G;
    w.r1 = min(w.r0 + tile_rows, w.n_rows);
    w.p_hi = o.p0 + (w.r1 - 1) / G;
    w.kb = key_blocks<S::KEYS>(a.c.window, a.c.sinks, w.p_lo, w.p_hi);
    w.of = key_splits(w.kb.total, splits);
    if (split >= w.of) {   // nothing left for it
        w.n_rows = w.r1 = 0;
        return w;
    }
    w.b0 = (int)((long long)w.kb.total * split / w.of);
    w.nb = (int)((long long)w.kb.total * (split + 1) / w.of) - w.b0;
    return w;
}

template <int DH, bool F16>
__global__ void __launch_bounds__(kPThreads, 1)
    paged_prompt_kernel(const __grid_constant__ PromptMaps maps, const PagedAttnArgs a, int most_tiles, bool may_split,
                        bool join_later) {
    using S = PromptShape<DH>;
    constexpr int ST = S::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* Qs = smem;                     // [halves][256 rows][128 B]
    uint8_t* ring = smem + S::QBYTES;       // [stages][halves][128 keys][128 B]
    __shared__ uint64_t full[ST], empty[ST], clean[ST / 2], work_ready[2], work_taken[2], q_ready[2], q_free, o_free[2], drained;
    __shared__ uint64_t s_full[S::TILES], p_ready[S::TILES], o_done[S::TILES];
    __shared__ uint32_t tmem_base, block_mapped[16];   // of block g at g % 16: at most ST / 2 are in the ring
    __shared__ uint32_t odd_piece[4];   // of piece t at t % 4: 8-dimension chunks of which values were taken out
    __shared__ TileOrder order;
    __shared__ PromptWork work[4];       // piece t at t % 4: written again when the rows are done with it
    __shared__ float top_x[S::ROWS], l_part[S::SHARES][S::ROWS];   // a row's highest score, between its threads; their sums

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int G = a.c.Hq / a.c.Hk, most = most_tiles * a.c.Hk + (int)gridDim.x;   // pieces at most
    pdl_trigger();
    if (tid == 0) {
        tma_prefetch_map(&maps.q);
        tma_prefetch_map(&maps.k);
        tma_prefetch_map(&maps.v);
        for (int s = 0; s < ST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < ST / 2; ++s) mbar_init(&clean[s], 1);   // values of block g at g % (ST / 2)
        mbar_init(&q_free, 1);
        mbar_init(&drained, 1);
        for (int i = 0; i < S::TILES; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 4 * S::SHARES);
            mbar_init(&o_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&work_ready[i], 1);
            mbar_init(&work_taken[i], 1);
            mbar_init(&q_ready[i], 1);
            mbar_init(&o_free[i], 16 + 1);
        }
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(&tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    pdl_wait();
    const bool ordered = !may_split && most_tiles <= kSortTiles && a.batch <= kSortTiles;
    if (ordered) order_tiles<S>(a, most_tiles, order);
    if (blockIdx.x == 0)   // reports every session whose indices do not fit
        for (int i = tid; i < a.batch; i += kPThreads) {
            AttnSession o;
            attn_session(a, i, o);
        }
    bool ok = true;   // false after a wait that gave up: no other waits any more, and what is computed is not used
    auto wait = [&](uint64_t* bar, int phase) {
        if (!ok) return;
        ok = __all_sync(0xffffffffu, mbar_poll(bar, (uint32_t)(phase & 1), kPollLimit) != 0);
        if (!ok && lane == 0) atomicOr(a.c.status, VC_DEV_TIMEOUT);
    };
    // Every role goes through the CTA's pieces in turn (t counts them, g the key blocks since the launch) and is held
    // up by barriers alone: the copies, the rows of Q and the first scores of a piece come while the one before ends.
    // No barrier completes twice before all that wait for it have seen it once: work_ready, q_ready and o_free alternate
    // (piece t + 2 is handed out after the copies' warp took piece t, which nothing else waits for where pieces have no
    // blocks; the products of piece t + 1 begin after o_free of t, and q_ready of t + 2 after those), the others are held
    // back by the arrivals of the same threads.

    // the rows' warps take registers that the other four give up; in each SM quarter 4 x 104 + 64 = 5 x 96, the launch's
    if (warp < 4) {
        set_registers<false, 64>();
        if (warp == 0) {
            // ---- copies: K of a block, V of the block, K of the next, ... in ring order ----
            const int box_rows = min(a.c.page, S::KEYS), boxes = S::KEYS / box_rows;
            int issued = 0;
            for (int t = 0; t <= most && ok; ++t) {
                wait(&work_ready[t & 1], t >> 1);
                const PromptWork w = work[t & 3];
                __syncwarp();
                if (lane == 0) mbar_arrive(&work_taken[t & 1]);
                if (w.nb < 0) break;
                int entry = -1;
                auto look_up = [&](int n) {   // lane q < boxes: the table entry of block n's q-th box
                    entry = -1;
                    const int t = n < w.nb ? w.kb.block(w.b0 + n) * S::KEYS + lane * box_rows : INT32_MAX;
                    if (lane < boxes && t <= w.p_hi) entry = page_of(a.c, w.s, t >> a.c.page_shift);
                };
                look_up(0);
                for (int n = 0; n < w.nb && ok; ++n) {
                    const int t = w.kb.block(w.b0 + n) * S::KEYS + lane * box_rows;
                    const bool there = entry >= 0;
                    const unsigned mapped = __ballot_sync(0xffffffffu, there);
                    const int pool_row = (entry * a.c.Hk + w.j) * a.c.page + (t & (a.c.page - 1));
                    look_up(n + 1);
                    for (int kv = 0; kv < 2; ++kv, ++issued) {
                        const int s = issued & (ST - 1);
                        if (issued >= ST) wait(&empty[s], issued / ST - 1);
                        if (!ok) break;
                        if (lane == 0) {
                            if (kv == 0) {   // a bit for each 16 keys
                                uint32_t groups = 0;
                                for (int u = 0; u < S::KEYS / 16; ++u) groups |= ((mapped >> (16 * u / box_rows)) & 1u) << u;
                                block_mapped[(issued >> 1) & 15] = groups;
                            }
                            mbar_arrive_expect_tx(&full[s], (uint32_t)(__popc(mapped) * box_rows * DH * 2));
                        }
                        __syncwarp();
                        if (there)
#pragma unroll
                            for (int h = 0; h < S::HALVES; ++h)
                                tma_load_2d(ring + s * S::TILE + h * (S::KEYS * 128) + lane * box_rows * 128, kv ? &maps.v : &maps.k,
                                            h * 64, pool_row, &full[s]);
                    }
                }
            }
            // no copy outlives the CTA: after a wait that gave up, each gets another bounded while
            if (!ok)
                for (int k = max(0, issued - ST); k < issued; ++k) mbar_wait(&full[k & (ST - 1)], (uint32_t)((k / ST) & 1), nullptr);
        } else if (warp == 1) {
            // ---- products ----
            constexpr uint32_t ID_S = umma_idesc(!F16, false, 128, S::KEYS), ID_O = umma_idesc(!F16, true, 128, DH);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            uint32_t fine = 1;
            const uint64_t q_desc = desc_sw128(smem_u32(Qs)), k_desc = desc_sw128(smem_u32(ring)),
                           v_desc = umma_desc(smem_u32(ring), S::KEYS * 128, 1024, UMMA_SW128);   // addresses count 16 bytes
            auto mma_s = [&](int i, int s) {   // S_i = Q_i K^T
#pragma unroll
                for (int c = 0; c < DH / 16; ++c) {
                    tc_mma(tm + S::S0 + (uint32_t)(i * S::KEYS),
                           q_desc + (uint32_t)((i * (128 * 128) + (c >> 2) * (S::ROWS * 128) + (c & 3) * 32) / 16),
                           k_desc + (uint32_t)s * (S::TILE / 16) + (uint32_t)(((c >> 2) * (S::KEYS * 128) + (c & 3) * 32) / 16), ID_S, c != 0);
                }
                tc_commit(&s_full[i]);
            };
            auto mma_o = [&](int i, int s, bool first) {   // O_i += P_i V
#pragma unroll
                for (int c = 0; c < S::KEYS / 16; ++c)
                    tc_mma_ta(tm + S::O0 + (uint32_t)(i * DH), tm + S::S0 + (uint32_t)(i * S::KEYS + (c >> 2) * 64 + (c & 3) * 8),
                              v_desc + (uint32_t)s * (S::TILE / 16) + (uint32_t)(c * 2048 / 16), ID_O, c != 0 || !first);
                tc_commit(&o_done[i]);
            };
            auto hold = [&](uint64_t* bar, int phase) {   // as wait(), with control flow that is the same in all lanes
                fine &= mbar_poll(bar, (uint32_t)(phase & 1), fine ? kPollLimit : 1u);
                __syncwarp();
            };
            auto slot = [](int k) { return k & (ST - 1); };
            int g = 0, gi[S::TILES];   // blocks so far, and those that a tile had rows for
#pragma unroll
            for (int i = 0; i < S::TILES; ++i) gi[i] = 0;
            for (int t = 0; t <= most; ++t) {
                hold(&q_ready[t & 1], t >> 1);
                const int nb = __shfl_sync(0xffffffffu, work[t & 3].nb, 0);
                const int used = __shfl_sync(0xffffffffu, (work[t & 3].r1 - work[t & 3].r0 + 127) >> 7, 0);   // tiles with rows
                if (nb < 0) break;
                if (nb > 0) {
                    hold(&full[slot(2 * g)], 2 * g / ST);
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < S::TILES; ++i)
                            if (i < used) mma_s(i, slot(2 * g));
                        tc_commit(&empty[slot(2 * g)]);
                    }
                    __syncwarp();
                    if (t > 0) hold(&o_free[(t - 1) & 1], (t - 1) >> 1);   // the outputs of the piece before were read
                    if (nb == 1) {
                        if (elect_one()) tc_commit(&q_free);
                        __syncwarp();
                    }
                } else {
                    if (t > 0) hold(&o_free[(t - 1) & 1], (t - 1) >> 1);
                    if (lane == 0) mbar_arrive(&q_free);
                    __syncwarp();
                }
                for (int n = 0; n < nb; ++n, ++g) {
                    const bool more = n + 1 < nb;
                    const int sv = slot(2 * g + 1), sk = slot(2 * g + 2);
                    hold(&clean[g & (ST / 2 - 1)], g / (ST / 2));   // the values are there and clean
                    if (more) hold(&full[sk], (2 * g + 2) / ST);
#pragma unroll
                    for (int i = 0; i < S::TILES; ++i) {
                        if (i >= used) continue;
                        hold(&p_ready[i], gi[i]);
                        ++gi[i];
                        tc_fence_after();
                        if (elect_one()) {
                            mma_o(i, sv, n == 0);
                            if (more) mma_s(i, sk);
                            if (i == used - 1) {
                                tc_commit(&empty[sv]);
                                if (more) tc_commit(&empty[sk]);
                                if (n + 2 == nb) tc_commit(&q_free);
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            if (!fine) {   // no product outlives the tensor memory
                if (lane == 0) {
                    atomicOr(a.c.status, VC_DEV_TIMEOUT);
                    tc_commit(&drained);
                }
                mbar_wait(&drained, 0, nullptr);
            }
        } else if (warp == 2) {
            // ---- the pieces, handed out as CTAs come for them (the first by index), and their rows of Q ----
            const int tiles = ordered ? order.count : count_tiles(a, G, S::ROWS / G * G, most_tiles), units = tiles * a.c.Hk;
            const int splits = may_split ? unit_splits(units, (int)gridDim.x) : 1, items = units * splits;
            int t = 0;
            for (; t <= most; ++t) {
                int item = blockIdx.x;
                if (t > 0) {
                    if (lane == 0) {
                        const int k = atomicAdd(a.ticket, 1);   // each CTA takes one behind the last piece: `items` in all
                        if (k == items - 1) *a.ticket = 0;
                        item = (int)gridDim.x + k;
                    }
                    item = __shfl_sync(0xffffffffu, item, 0);
                }
                const PromptWork w = prompt_work<S>(a, ordered ? &order : nullptr, tiles, splits, item);
                if (t > 1) wait(&work_taken[t & 1], (t - 2) >> 1);
                if (lane == 0) {
                    work[t & 3] = w;
                    odd_piece[t & 3] = 0;
                    mbar_arrive(&work_ready[t & 1]);
                }
                if (t > 0) wait(&q_free, t - 1);   // the scores of the piece before are complete
                if (lane == 0) {
                    if (w.nb > 0 && ok) {
                        mbar_arrive_expect_tx(&q_ready[t & 1], (uint32_t)(S::ROWS / G * G * DH * 2));
                        for (int h = 0; h < S::HALVES; ++h)
                            for (int k = 0; k < S::ROWS / G; k += 256)   // tokens of a box (more than one where G is 1)
                                tma_load_3d(Qs + (h * S::ROWS + k) * 128, &maps.q, h * 64, w.j * G, w.row0 + w.r0 / G + k,
                                            &q_ready[t & 1]);
                    } else {
                        mbar_arrive(&q_ready[t & 1]);
                    }
                }
                __syncwarp();
                if (w.nb < 0) break;
            }
            // no rows of Q on their way outlive the CTA: these have come, unless a wait gave up (then a bounded while more)
            for (int b = max(t - 1, 0); b <= t; ++b) mbar_poll(&q_ready[b & 1], (uint32_t)((b >> 1) & 1), kPollLimit);
        } else if (warp == 3) {
            // ---- values that not every row of the tile sees: those that no row sees become 0, and so do infinities and
            // NaN (the rows that see them get them at the end), so that a weight of 0 takes nothing in ----
            int g = 0;
            for (int t = 0; t <= most; ++t) {
                wait(&q_ready[t & 1], t >> 1);
                const PromptWork w = work[t & 3];
                if (w.nb < 0) break;
                for (int n = 0; n < w.nb; ++n, ++g) {
                    const int s = (2 * g + 1) & (ST - 1), t0 = w.kb.block(w.b0 + n) * S::KEYS;
                    wait(&full[s], (2 * g + 1) / ST);
                    const uint32_t groups = block_mapped[g & 15];
                    const bool whole = groups == S::ALL && t0 + S::KEYS - 1 <= w.p_lo &&
                                       (a.c.window == 0 || t0 > w.p_hi - a.c.window || t0 + S::KEYS - 1 < a.c.sinks);
                    if (!whole && ok) {
                        uint8_t* Vs = ring + s * S::TILE;
                        constexpr int ROW = S::HALVES * 8;   // 16-byte chunks of a row (their order does not matter)
                        uint32_t odd = 0;   // chunks of 8 dimensions
                        // rows first .. last - 1 of the block: seen by none, or by some
                        auto sweep = [&](int first, int last, bool none) {
                            const int n_chunks = max(last - first, 0) * ROW;
#pragma unroll 4
                            for (int k = lane; k < n_chunks; k += 32) {
                                const int c = k % ROW;
                                uint4* at = reinterpret_cast<uint4*>(Vs + (c >> 3) * (S::KEYS * 128) + (first + k / ROW) * 128 + (c & 7) * 16);
                                if (none) {
                                    *at = make_uint4(0u, 0u, 0u, 0u);
                                } else {
                                    const uint4 x = *at;
                                    if (any_nonfinite<F16>(x)) {
                                        odd |= 1u << ((c & 8) | ((c ^ (first + k / ROW)) & 7));   // (swizzled rows)
                                        *at = make_uint4(finite2<F16>(x.x), finite2<F16>(x.y), finite2<F16>(x.z), finite2<F16>(x.w));
                                    }
                                }
                            }
                            __syncwarp();
                        };
                        auto clip = [&](long long at) { return (int)(at < t0 ? 0 : at > t0 + S::KEYS ? S::KEYS : at - t0); };
                        // no page: whatever an earlier block left there
                        for (int u = 0; u < S::KEYS / 16; ++u)
                            if (!((groups >> u) & 1u)) sweep(16 * u, 16 * u + 16, true);
                        sweep(clip(w.p_lo + 1LL), clip(w.p_hi + 1LL), false);   // the first row sees up to p_lo, the last to p_hi
                        sweep(clip(w.p_hi + 1LL), S::KEYS, true);
                        if (a.c.window > 0) {                                    // and from p_lo - window + 1 on, behind the sinks
                            const long long from = w.p_lo - (long long)a.c.window + 1, to = w.p_hi - (long long)a.c.window + 1;
                            sweep(clip(a.c.sinks), clip(from), true);
                            sweep(clip(from > a.c.sinks ? from : a.c.sinks), clip(to), false);
                        }
                        if (odd) atomicOr(&odd_piece[t & 3], odd);
                        fence_proxy_async();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&clean[g & (ST / 2 - 1)]);
                }
                if (lane == 0) mbar_arrive(&o_free[t & 1]);   // this role is done with the piece, too
            }
        }
        set_registers<true, 96>();
    } else {
        set_registers<true, 104>();
        // ---- rows: a row's scores of a block belong to one thread or two (64 each).  The warps of an SM quarter, four
        // tiles' or two tiles' with two shares each, take turns at its special function units ----
        const int i = (warp - 4) / (4 * S::SHARES), half = ((warp - 4) >> 2) % S::SHARES, quarter = warp & 3, rr = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + lanes + S::S0 + (uint32_t)(i * S::KEYS + half * 64), tO = tmem + lanes + S::O0 + (uint32_t)(i * DH);
        const int pair = 1 + i * 4 + quarter;   // the barrier of a row's two warps
        const float2 by = make_float2(a.scale_log2, a.scale_log2);
        int gi = 0;   // blocks so far for this tile
        int g = 0;
        for (int t = 0; t <= most; ++t) {
            wait(&q_ready[t & 1], t >> 1);
            const PromptWork& w = work[t & 3];
            const int n_all = w.nb, r = w.r0 + i * 128 + rr;
            if (n_all < 0) break;
            const int nb = w.r0 + i * 128 < w.r1 ? n_all : 0;   // a tile without rows has nothing to do
            const bool in = r < w.r1;   // rows behind the tile's last decide nothing (whatever their Q is)
            const PromptRow me{w.p0 + r / G, a.c.window, a.c.sinks};
            const int w_lo = w.p0 + (r - lane) / G, w_hi = w.p0 + (r - lane + 31) / G;   // the warp's rows
            // m: the maximum under which the row's weights stand (its threads agree on it); l: the sum of this thread's
            float m = -INFINITY, l = 0.0f;
            for (int n = 0; n < nb; ++n, ++gi) {
                const int t0 = w.kb.block(w.b0 + n) * S::KEYS + half * 64;
                const bool inside = t0 + 63 <= w_lo && (a.c.window == 0 || t0 > w_hi - a.c.window || t0 + 63 < a.c.sinks);
                const bool standing = __all_sync(0xffffffffu, m != -INFINITY || !in);   // of the same rows in both warps
                wait(&s_full[i], gi);
                tc_fence_after();
                const uint32_t groups = block_mapped[(g + n) & 15] >> (4 * half);
                const bool whole = inside && (groups & 0xfu) == 0xfu;
                float v[32];
                float2 part[2];
                uint32_t pk[2][16];
                auto take = [&](int c) {   // scores of columns c .. c + 31, -inf where not seen
                    tc_ld32(tS + (uint32_t)c, v);
                    if (!whole) {
                        const uint32_t seen = me.seen(t0 + c, groups >> (c >> 4));
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = (seen >> e) & 1u ? v[e] : -INFINITY;
                    }
                };
                // the weights 2^(z scale - base): added to the sum, and rounded to 16 bits as the tensor core takes them
                // (up to 2^-8 of a weight in bf16, 2^-11 in fp16); 0 where not seen
                auto weigh = [&](uint32_t (&u)[16], float2 off) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 z = fma2(make_float2(v[2 * e], v[2 * e + 1]), by, off);
                        z.x = exp2_approx(z.x);
                        z.y = exp2_approx(z.y);
                        part[e & 1] = add2(part[e & 1], z);
                        u[e] = pack16<F16>(z.x, z.y);
                    }
                };
                auto weigh_all = [&](float base) {   // one pass over the thread's scores -> the sum of its weights
                    const float2 off = make_float2(-base, -base);
                    part[0] = part[1] = make_float2(0.0f, 0.0f);
                    take(0);
                    weigh(pk[0], off);
                    take(32);
                    weigh(pk[1], off);
                    return (part[0].x + part[0].y) + (part[1].x + part[1].y);
                };
                // The weights under the maximum that stands, which holds nearly always: a sum of at most 2^14 has no weight
                // above it, which both 16-bit types hold.  (64 weights of at most 2^8 do not pass it.)
                float sum = 0.0f;
                if (standing) sum = weigh_all(m);
                const bool grew = in && !(sum <= 16384.0f);   // or a score is not a number
                if (!standing || (S::SHARES == 2 ? any_of_pair(pair, grew) : __any_sync(0xffffffffu, grew))) {
                    // it moves where it grew by more than 8 (a factor of 2^8), or was none (then all weights so far were 0)
                    float t4[4];
                    t4[0] = t4[1] = t4[2] = t4[3] = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 64; c += 32) {
                        take(c);
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
#pragma unroll
                            for (int u = 0; u < 4; ++u) t4[u] = max3(t4[u], v[e + u], v[e + 4 + u]);
                    }
                    float tp = max3(t4[0], max3(t4[1], t4[2], t4[3]), t4[3]) * a.scale_log2;   // scale above 0
                    if (S::SHARES == 2) {
                        float& x = top_x[i * 128 + rr];
                        if (half == 0) x = tp;
                        sync_pair(pair);
                        if (half == 1) x = max3(tp, x, tp);
                        sync_pair(pair);
                        tp = x;
                    }
                    const float m_new = tp <= m + 8.0f ? m : tp;   // NaN moves it too, and makes the row's sum NaN
                    const float f = !in || m == -INFINITY || m_new == m ? 1.0f : exp2_approx(m - m_new);
                    m = m_new;
                    l *= f;
                    if (n > 0 && __any_sync(0xffffffffu, f != 1.0f)) {   // the products so far are in O_i; the row's threads share its columns
                        wait(&o_done[i], gi - 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = half * (DH / S::SHARES); c < (half + 1) * (DH / S::SHARES); c += 16) {
                            float x[16];
                            tc_ld16(tO + (uint32_t)c, x);
                            uint32_t u[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(x[e] * f);
                            tc_st16(tO + (uint32_t)c, u);
                        }
                    }
                    sum = weigh_all(m == -INFINITY ? 0.0f : m);
                }
                l += sum;
                tc_st16(tS, pk[0]);
                tc_st16(tS + 16, pk[1]);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[i]);   // (arrivals of all lanes would take turns)
            }
            // ---- out, or a split's record: [ROWS][DH] sums, [ROWS] maxima, [ROWS] sums of weights ----
            if (nb > 0) {
                if (S::SHARES == 2) {
                    l_part[half][i * 128 + rr] = l;
                    sync_pair(pair);
                    l = l_part[0][i * 128 + rr] + l_part[S::SHARES - 1][i * 128 + rr];
                }
            }
            const int at = i * 128 + rr;
            const long long mine = in ? (long long)(w.row0 + r / G) * a.out_ld + (long long)(w.j * G + r % G) * DH : -1;
            long long to[4];   // where the rows of the thread's group of four go
#pragma unroll
            for (int u = 0; u < 4; ++u) to[u] = __shfl_sync(0xffffffffu, mine, (lane & ~3) + u);
            const int of = w.of;
            const float inv = of > 1 ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
            float* rec = a.partial + (size_t)w.record * (S::ROWS * (DH + 2));
            if (nb > 0) {
                wait(&o_done[i], gi - 1);
                tc_fence_after();
            }
            // bits: chunks of 8 dimensions with infinities or NaN, taken out of the values or in the thread's results
            uint32_t odd = odd_piece[t & 3];
#pragma unroll 1
            for (int c = half * (DH / S::SHARES); c < (half + 1) * (DH / S::SHARES); c += 32) {
                float v[32];
                if (nb > 0) tc_ld32(tO + (uint32_t)c, v);
                else
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.0f;
                if (c + 32 == (half + 1) * (DH / S::SHARES)) {   // O_i may be written again
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&o_free[t & 1]);
                }
                if (!ok) continue;
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] *= inv;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float x = v[8 * k] * 0.0f;
#pragma unroll
                    for (int e = 1; e < 8; ++e) x = fmaf(v[8 * k + e], 0.0f, x);
                    if (x != 0.0f) odd |= 1u << (c / 8 + k);
                }
                if (of == 1) {
                    // four lanes exchange the 16-byte pieces of their rows, so that each writes 64 bytes of a row together
                    uint4 x[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        x[u] = make_uint4(pack_out<F16>(a.widen, v[8 * u], v[8 * u + 1]),
                                          pack_out<F16>(a.widen, v[8 * u + 2], v[8 * u + 3]),
                                          pack_out<F16>(a.widen, v[8 * u + 4], v[8 * u + 5]),
                                          pack_out<F16>(a.widen, v[8 * u + 6], v[8 * u + 7]));
                    swap_lanes(x[0], x[1], 1, lane & 1);
                    swap_lanes(x[2], x[3], 1, lane & 1);
                    swap_lanes(x[0], x[2], 2, lane & 2);
                    swap_lanes(x[1], x[3], 2, lane & 2);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (to[u] >= 0) *reinterpret_cast<uint4*>(a.out + to[u] + c + (lane & 3) * 8) = x[u];
                } else if (in) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        __stcg(reinterpret_cast<float4*>(rec + at * DH + c + e), make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
                }
            }
            if (__any_sync(0xffffffffu, odd != 0)) {   // the rows that see them get them
                __threadfence_block();
                __syncwarp();   // (lanes write one another's rows)
                if (in && ok && l == l) {
                    const SeenValues<DH> values = seen_values<DH>(a.c, w.s, w.j, me.p);
#pragma unroll 1
                    for (int d = half * (DH / S::SHARES); d < (half + 1) * (DH / S::SHARES); d += 4) {
                        if (!((odd >> (d / 8)) & 1u)) continue;
                        const float4 z = odd_values<DH, F16>(values, d);
                        float* r4 = rec + at * DH + d;
                        uint16_t* o4 = a.out + mine + d;
                        auto put = [&](int u, float x) {
                            if (x == 0.0f) return;
                            if (of > 1) __stcg(r4 + u, x);
                            else o4[u] = (uint16_t)pack_out<F16>(a.widen, x, 0.0f);
                        };
                        put(0, z.x); put(1, z.y); put(2, z.z); put(3, z.w);
                    }
                }
            }
            if (of > 1 && half == 0 && in) {
                __stcg(rec + S::ROWS * DH + at, m);
                __stcg(rec + S::ROWS * DH + S::ROWS + at, l);
            }
            g += n_all;
        }
        set_registers<false, 96>();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    const PromptWork& w = work[0];   // a CTA has one piece where tiles are split
    if (!may_split || join_later || w.n_rows == 0 || w.of <= 1) return;
    if (!last_to_arrive(a.merge + w.record / w.splits, w.of)) return;
    const int first = w.row0 * G + w.r0;   // packed rows of the whole call
    join_records<DH, F16, kPThreads>(a, a.partial + (size_t)(w.record - w.record % w.splits) * (S::ROWS * (DH + 2)), S::ROWS, w.of,
                                     0, w.r1 - w.r0, reinterpret_cast<float*>(smem), [&](int r) {
                                         return a.out + (size_t)((first + r) / G) * a.out_ld + (size_t)(w.j * G + (first + r) % G) * DH;
                                     }, [&](int r, int d) { return odd_values<DH, F16>(seen_values<DH>(a.c, w.s, w.j, w.p0 + (w.r0 + r) / G), d); });
}

template <int DH, bool F16>
static cudaError_t launch_prompts_t(const PagedAttnArgs& a, cudaStream_t s) {
    using S = PromptShape<DH>;
    const long long G = a.c.Hq / a.c.Hk;
    if (G > 256) return cudaErrorNotSupported;
    // at most: every session's last tile may be part-filled
    const long long tile_rows = S::ROWS / G * G, tiles = (a.rows * G + tile_rows - 1) / tile_rows + a.batch,
                    units = tiles * a.c.Hk;
    if (units > INT32_MAX - kMaxSms) return cudaErrorNotSupported;
    // the key blocks are split where that gives more SMs work
    const bool may_split = (a.rows * G + tile_rows - 1) / tile_rows * a.c.Hk * 2 <= a.num_sms, join_later = may_split && many_keys(a);
    static_assert(S::BYTES - 1024 >= kMostSplits * S::ROWS * 4, "room for the join's factors");
    PromptMaps maps;
    const int rows = a.c.pages * a.c.Hk * a.c.page, box = a.c.page < S::KEYS ? a.c.page : S::KEYS;
    EncodeTiledFn encode = tma_encode_fn();
    // a tile's rows of Q: whole tokens, the heads of one KV head of each, packed as they come
    const cuuint64_t dims[3] = {(cuuint64_t)DH, (cuuint64_t)a.c.Hq, (cuuint64_t)a.rows};
    const cuuint64_t strides[2] = {(cuuint64_t)DH * 2, (cuuint64_t)a.q_ld * 2};
    const cuuint32_t q_box[3] = {64, (cuuint32_t)G, (cuuint32_t)(S::ROWS / G < 256 ? S::ROWS / G : 256)}, unit[3] = {1, 1, 1};
    if (!encode ||
        encode(&maps.q, F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(a.q),
               dims, strides, q_box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
        !tma_map_2d(&maps.k, a.c.k, rows, DH, DH, 64, box, F16, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !tma_map_2d(&maps.v, a.c.v, rows, DH, DH, 64, box, F16, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    auto kern = paged_prompt_kernel<DH, F16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(!may_split && units < a.num_sms ? units : a.num_sms));
    cfg.blockDim = dim3(kPThreads);
    cfg.dynamicSmemBytes = S::BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = a.pdl;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, maps, a, (int)tiles, may_split, join_later);
    return e == cudaSuccess && join_later
               ? launch_paged_join(a, JoinShape{S::ROWS, (int)tile_rows, S::KEYS, (int)tiles, a.num_sms}, s)
               : e;
}

cudaError_t launch_paged_prompts(const PagedAttnArgs& a, cudaStream_t s) {
    if (!(a.scale_log2 > 0.0f)) return cudaErrorNotSupported;   // the row maximum is taken before the scale
    if (a.c.Dh == 128) return a.f16 ? launch_prompts_t<128, true>(a, s) : launch_prompts_t<128, false>(a, s);
    if (a.c.Dh == 64) return a.f16 ? launch_prompts_t<64, true>(a, s) : launch_prompts_t<64, false>(a, s);
    return cudaErrorNotSupported;
}

}  // namespace vc
