// paged_frame.cu -- windowed attention over the paged KV cache for single frames (one row per session).
//
// Bound: HBM.  A frame reads min(ctx, window + sinks) keys and values per session and KV head once, 4 Dh bytes
// each, and does 4 G Dh flops on them (G = q_heads / kv_heads query heads share them).
//
// The work of all sessions is one line of units (session, KV head, block of BK keys), cut into equal ranges, one
// CTA per SM: however ragged the sessions are, every SM reads the same amount.  In a CTA the units go round the
// warps; each warp keeps a ring of TMA copies ahead of it (K and V blocks, swizzled rows, fetched page by
// page through the table) and its own running maximum, sum and output of the softmax in registers.  The products
// run on warp-level matrix instructions with the keys (then the head dims) as the 16 rows and the query heads as
// the 8 columns, S^T = K Q^T and O^T = V^T P^T: up to 8 heads waste no row, and P^T is S^T's registers transposed.
// At the end of a (session, KV head) the warps join through shared memory; where a range ends inside one, the
// CTAs that share it leave records, and the last of them to arrive joins these in order, so that results do not
// depend on timing.
// The weights go into the products as a 16-bit value and the 16-bit rest of it: the error of a weight is
// 2^-16 (bf16), and the products are not what this kernel waits for.
#include "paged_dev.cuh"
#include "tc.cuh"

namespace vc {

static constexpr int kFMaxStages = 4;
static constexpr int kFMaxBatch = 2048;

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
    const int comb = S::WARPS * G * (S::CS + 2) * 4, weights = grid * (2 * G + 1) * 4, sessions = (batch + 1) * 16;
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
    float* comb = reinterpret_cast<float*>(smem + L.off_comb);        // [warps][G][CS], then [warps][G][2]
    float* wts = reinterpret_cast<float*>(smem + L.off_weights);      // [CTAs][G][2], then [CTAs] records
    LineSession* line = reinterpret_cast<LineSession*>(smem + L.off_sessions);   // [batch + 1]
    __shared__ uint64_t full[kWarps][kFMaxStages];
    __shared__ uint32_t stage_mapped[kWarps][kFMaxStages];
    __shared__ int warp_total[kWarps], last_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
    const int G = a.c.Hq / a.c.Hk, Hk = a.c.Hk;
    if (lane == 0)
        for (int s = 0; s < L.stages; ++s) mbar_init(&full[warp][s], 1);
    fence_mbar_init();

    // the line's sessions (every CTA lays out the same line)
    int units = 0;
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
        if (lane == 31) warp_total[warp] = incl;
        __syncthreads();
        int before = units;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += warp_total[w];
            units += warp_total[w];
        }
        me.first = before + incl - me.blocks * Hk;
        if (b < a.batch) line[b] = me;
        __syncthreads();
    }
    if (tid == 0) line[a.batch] = LineSession{units, 0, 0, 0};
    __syncthreads();
    if (units == 0) return;

    const long long grid = min((int)gridDim.x, units);   // ranges, none of them empty
    if (blockIdx.x >= grid) return;
    auto range_start = [&](long long c) { return (int)(c * units / grid); };
    auto owner = [&](int x) { return (int)((((long long)x + 1) * grid - 1) / units); };
    const int c0 = range_start(blockIdx.x), c1 = range_start(blockIdx.x + 1);

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
    Place here{0, 0, 0};   // the CTA's first unit
    {
        int lo = 0, hi = a.batch - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (line[mid].first <= c0) lo = mid;
            else hi = mid - 1;
        }
        const int rel = c0 - line[lo].first, n = line[lo].blocks;
        here = Place{lo, rel / n, rel % n};
    }

    // ---- this warp's copies: unit c0 + warp + WARPS i is copy i, in ring slot i % stages ----
    uint8_t* ring = smem + (size_t)warp * L.stages * S::STAGE;
    const int box_rows = min(a.c.page, BK), boxes = BK / box_rows;
    int copy_x = c0 + warp, copy_slot = 0, look_x = copy_x, issued = 0;
    Place look = here;
    if (look_x < c1) forward(look, warp);
    // looks up the pages of the next copy but those looked up before; lane q < boxes gets the pool row of its q-th
    // box, -1: no page
    auto look_up = [&]() {
        int pool_row = -1;
        if (look_x < c1) {
            const LineSession me = line[look.b];
            const KeyBlocks kb = key_blocks<BK>(a.c.window, a.c.sinks, me.p, me.p);
            const int t = kb.block(look.blk) * BK + lane * box_rows;
            if (lane < boxes && t <= me.p) {
                const int e = page_of(a.c, me.s, t >> a.c.page_shift);
                if (e >= 0) pool_row = (e * Hk + look.j) * a.c.page + (t & (a.c.page - 1));
            }
            look_x += kWarps;
            if (look_x < c1) forward(look, kWarps);
        }
        return pool_row;
    };
    auto issue = [&](int pool_row) {   // starts the copy of a look-up, in order
        if (copy_x >= c1) return;
        const unsigned mapped = __ballot_sync(0xffffffffu, pool_row >= 0);
        uint64_t* bar = &full[warp][copy_slot];
        if (lane == 0) {
            stage_mapped[warp][copy_slot] = mapped;
            mbar_arrive_expect_tx(bar, (uint32_t)(__popc(mapped) * box_rows * DH * 4));
        }
        __syncwarp();
        if (pool_row >= 0) {
            uint8_t* to = ring + copy_slot * S::STAGE + lane * box_rows * S::ROWB;
#pragma unroll
            for (int part = 0; part < S::PARTS; ++part) {
                tma_load_2d(to + part * (BK * 128), &tmK, part * 64, pool_row, bar);
                tma_load_2d(to + S::KBYTES + part * (BK * 128), &tmV, part * 64, pool_row, bar);
            }
        }
        copy_x += kWarps;
        copy_slot = copy_slot + 1 == L.stages ? 0 : copy_slot + 1;
        ++issued;
    };
    {
        int rows[kFMaxStages];   // the first copies' table reads are in flight together
#pragma unroll
        for (int s = 0; s < kFMaxStages; ++s)
            if (s < L.stages) rows[s] = look_up();
#pragma unroll
        for (int s = 0; s < kFMaxStages; ++s)
            if (s < L.stages) issue(rows[s]);
    }
    int next_row = look_up();   // read while the warp computes

    // ---- units ----
    int slot = 0, phase = 0, used = 0;
    bool alive = true;   // false after a copy that never came: nothing more is computed, the barriers are kept
    const int mi = lane >> 3, lr = lane & 7;
    int x_seg = c0;
    while (x_seg < c1) {
        const Place at0 = here;   // of unit x_seg
        const int b = at0.b;
        const LineSession me = line[b];
        const int s0 = me.first + at0.j * me.blocks, s1 = s0 + me.blocks, end = min(s1, c1);
        const KeyBlocks kb = key_blocks<BK>(a.c.window, a.c.sinks, me.p, me.p);
        const int row = a.cu_rows ? a.cu_rows[b] : b;
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

        // the first unit from x_seg on that is this warp's
        static_assert((kWarps & (kWarps - 1)) == 0, "a power of two");
        int x = x_seg + ((warp - (x_seg - c0)) & (kWarps - 1));
        for (; x < end; x += kWarps) {
            ++used;
            if (alive) {
                alive = __all_sync(0xffffffffu, mbar_wait(&full[warp][slot], phase, a.c.status));
                if (!alive)   // the copies behind it are given another bounded while before anyone leaves
                    for (int k = used, sl = slot, ph = phase; k < issued; ++k) {
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
                    if (newest && seen(p - t0) && lane < S::CH) {   // the new row, to its page and into the block
                        const uint4 kv = *reinterpret_cast<const uint4*>(a.kn + (size_t)row * a.k_ld + at0.j * DH + lane * 8);
                        const uint4 vv = *reinterpret_cast<const uint4*>(a.vn + (size_t)row * a.v_ld + at0.j * DH + lane * 8);
                        const int e = page_of(a.c, me.s, p >> a.c.page_shift);
                        if (e >= 0) {
                            const size_t to = (((size_t)e * Hk + at0.j) * a.c.page + (p & (a.c.page - 1))) * DH + lane * 8;
                            *reinterpret_cast<uint4*>(a.c.k + to) = kv;
                            *reinterpret_cast<uint4*>(a.c.v + to) = vv;
                        }
                        *reinterpret_cast<uint4*>(Ks + S::at(p - t0, lane)) = kv;
                        *reinterpret_cast<uint4*>(Vs + S::at(p - t0, lane)) = vv;
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
                issue(next_row);
                next_row = look_up();
            }
            if (++slot == L.stages) {
                slot = 0;
                phase ^= 1;
            }
        }
        // ---- the warps' parts of this (session, KV head) ----
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[h][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int r = 8 * h + 2 * tq + e;
                if (r < G) {
                    float* rec = comb + (size_t)(warp * G + r) * CS;
                    if (sum != 0.0f)
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            rec[16 * mt + g] = acc[mt][h][e];
                            rec[16 * mt + g + 8] = acc[mt][h][2 + e];
                        }
                    if (g == 0) {
                        float* ml = comb + (size_t)kWarps * G * CS + (size_t)(warp * G + r) * 2;
                        ml[0] = m[h][e];
                        ml[1] = sum;
                    }
                }
            }
        __syncthreads();
        const bool shared_seg = s0 < c0 || s1 > c1;
        const int rec_floats = (G * (DH + 2) + 3) & ~3;   // 16-byte aligned records
        float* rec = a.partial + (size_t)(2 * blockIdx.x + (s0 <= c0 ? 0 : 1)) * rec_floats;
        const float* ml = comb + (size_t)kWarps * G * CS;
        auto out_at = [&](int r, int d) { return a.out + (size_t)row * a.out_ld + (size_t)(at0.j * G + r) * DH + d; };
        for (int i = tid; i < G * (DH / 4); i += kThreads) {
            const int r = i / (DH / 4), d = 4 * (i % (DH / 4));
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[(w * G + r) * 2]);
            const float base = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float lw = ml[(w * G + r) * 2 + 1];
                if (lw == 0.0f) continue;
                const float f = exp2_approx(ml[(w * G + r) * 2] - base);
                const float4 y = *reinterpret_cast<const float4*>(comb + ((size_t)w * G + r) * CS + d);
                sum = fmaf(lw, f, sum);
                v[0] = fmaf(y.x, f, v[0]); v[1] = fmaf(y.y, f, v[1]);
                v[2] = fmaf(y.z, f, v[2]); v[3] = fmaf(y.w, f, v[3]);
            }
            if (!shared_seg) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                *reinterpret_cast<uint2*>(out_at(r, d)) =
                    make_uint2(pack16<F16>(v[0] * inv, v[1] * inv), pack16<F16>(v[2] * inv, v[3] * inv));
            } else {
                __stcg(reinterpret_cast<float4*>(rec + r * DH + d), make_float4(v[0], v[1], v[2], v[3]));
                if (d == 0) __stcg(reinterpret_cast<float2*>(rec + G * DH + 2 * r), make_float2(top, sum));
            }
        }
        if (shared_seg) {
            __threadfence();
            __syncthreads();
            const int f = owner(s0), n = owner(s1 - 1) - f + 1;
            if (tid == 0) {
                last_flag = atomicAdd(a.merge + f, 1) == n - 1;
                if (last_flag) a.merge[f] = 0;
            }
            __syncthreads();
            if (last_flag) {
                __threadfence();
                // wts[k][r]: the k-th contributor's (maximum, sum), then its factor; its record is that of its first
                // segment if this one began at or before its range
                int* rec_at = reinterpret_cast<int*>(wts + 2 * n * G);
                for (int k = tid; k < n; k += kThreads)
                    rec_at[k] = (2 * (f + k) + (s0 <= range_start(f + k) ? 0 : 1)) * rec_floats;
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
                        if (w[1] != 0.0f) sum = fmaf(w[1], f2, sum);   // 0: a part without a key that is seen
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
                    *reinterpret_cast<uint2*>(out_at(r, d)) = make_uint2(pack16<F16>(v[0], v[1]), pack16<F16>(v[2], v[3]));
                }
            }
        }
        __syncthreads();
        if (end < c1) forward(here, end - x_seg);
        x_seg = end;
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
    kern<<<grid, S::THREADS, L.total, s>>>(mk, mv, a, L);
    return cudaGetLastError();
}

cudaError_t launch_paged_frames(const PagedAttnArgs& a, cudaStream_t s) {
    // a line of units that 32 bits count, in blocks of at least 16 keys; up to 16 query heads to a KV head (the rows
    // of one matrix instruction); sessions that the line's table in shared memory holds
    const long long most = (long long)a.c.columns * a.c.page / 16 + 2;
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
