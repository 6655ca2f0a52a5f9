// paged_frame.cu -- windowed attention over the paged KV cache for single frames (one row per session).
//
// Bound: HBM.  A frame reads min(ctx, window + sinks) keys and values per session and KV head once, 4 Dh bytes
// each, and does 4 G Dh flops on them (G = q_heads / kv_heads query heads share them).
//
// The work of all sessions is one line of units (session, KV head, block of BK keys), cut into equal ranges, one
// CTA per SM: however ragged the sessions are, every SM reads the same amount.  In a CTA the units go round the
// four warps; each warp keeps a ring of TMA copies ahead of it (K and V blocks, swizzled rows, fetched page by
// page through the table) and its own running maximum, sum and output of the softmax in registers, on
// warp-level matrix instructions with the G query heads as the 16 rows.  At the end of a (session, KV head) the
// four warps join through shared memory; where a range ends inside one, the CTAs that share it leave records,
// and the last of them to arrive joins these in order, so that results do not depend on timing.
// The weights go into the products as a 16-bit value and the 16-bit rest of it: the error of a weight is
// 2^-16 (bf16), and the products are not what this kernel waits for.
#include "paged_dev.cuh"
#include "tc.cuh"

namespace vc {

static constexpr int kFWarps = 4, kFThreads = 32 * kFWarps, kFMaxStages = 4;
static constexpr int kFMaxBatch = 2048;

template <int DH>
struct FrameShape {
    static constexpr int BK = DH >= 256 ? 16 : DH == 128 ? 32 : 64;   // keys per unit
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
    const int comb = kFWarps * G * (DH + 2) * 4, weights = (grid + 1) * G * 4, sessions = (batch + 1) * 16;
    const int rest = comb + weights + sessions + 1024 + 64;
    L.stages = (227 * 1024 - rest - 512) / (kFWarps * S::STAGE);
    if (L.stages > kFMaxStages) L.stages = kFMaxStages;
    L.off_comb = kFWarps * L.stages * S::STAGE;
    L.off_weights = L.off_comb + comb;
    L.off_sessions = (L.off_weights + weights + 15) / 16 * 16;
    L.total = (size_t)L.off_sessions + sessions + 1024;
    return L;
}

// a session of the line: its first unit, blocks per KV head, index in the cache, the row's position
struct LineSession {
    int first, blocks, s, p;
};

template <int DH, bool F16>
__global__ void __launch_bounds__(kFThreads, 1)
    paged_frame_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const PagedAttnArgs a, const FrameLayout L) {
    using S = FrameShape<DH>;
    constexpr int BK = S::BK, NT = DH / 8;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* comb = reinterpret_cast<float*>(smem + L.off_comb);        // [warps][G][DH], then [warps][G][2]
    float* wts = reinterpret_cast<float*>(smem + L.off_weights);      // [CTAs + 1][G]
    LineSession* line = reinterpret_cast<LineSession*>(smem + L.off_sessions);   // [batch + 1]
    __shared__ uint64_t full[kFWarps][kFMaxStages];
    __shared__ uint32_t stage_mapped[kFWarps][kFMaxStages];
    __shared__ int warp_total[kFWarps], last_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
    const int G = a.c.Hq / a.c.Hk, Hk = a.c.Hk;
    if (lane == 0)
        for (int s = 0; s < L.stages; ++s) mbar_init(&full[warp][s], 1);
    fence_mbar_init();

    // the line's sessions (every CTA lays out the same line)
    int units = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kFThreads) {
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
        for (int w = 0; w < kFWarps; ++w) {
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

    // a place on the line: unit x is block `blk` of session b's KV head j
    struct Place {
        int b, j, blk;
    };
    auto place = [&](int x, int b) {   // b: a session at or before x's
        while (x >= line[b + 1].first) ++b;
        const int rel = x - line[b].first, n = line[b].blocks;
        const int j = rel / n;
        return Place{b, j, rel - j * n};
    };
    int b_first = 0;
    {   // the session of the CTA's first unit
        int lo = 0, hi = a.batch - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (line[mid].first <= c0) lo = mid;
            else hi = mid - 1;
        }
        b_first = lo;
    }

    // ---- this warp's copies: unit c0 + warp + 4 i is copy i, in ring slot i % stages ----
    uint8_t* ring = smem + (size_t)warp * L.stages * S::STAGE;
    const int box_rows = min(a.c.page, BK), boxes = BK / box_rows;
    int copy_x = c0 + warp, copy_slot = 0, look_x = copy_x, look_b = b_first, issued = 0;
    // looks up the pages of the next copy but those looked up before; lane q < boxes gets the pool row of its q-th
    // box, -1: no page
    auto look_up = [&]() {
        int pool_row = -1;
        if (look_x < c1) {
            const Place u = place(look_x, look_b);
            look_b = u.b;
            const LineSession me = line[u.b];
            const KeyBlocks kb = key_blocks<BK>(a.c.window, a.c.sinks, me.p, me.p);
            const int t = kb.block(u.blk) * BK + lane * box_rows;
            if (lane < boxes && t <= me.p) {
                const int e = page_of(a.c, me.s, t >> a.c.page_shift);
                if (e >= 0) pool_row = (e * Hk + u.j) * a.c.page + (t & (a.c.page - 1));
            }
            look_x += kFWarps;
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
        copy_x += kFWarps;
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
    int b = b_first, x_seg = c0;
    while (x_seg < c1) {
        const Place at0 = place(x_seg, b);
        b = at0.b;
        const LineSession me = line[b];
        const int s0 = me.first + at0.j * me.blocks, s1 = s0 + me.blocks, end = min(s1, c1);
        const KeyBlocks kb = key_blocks<BK>(a.c.window, a.c.sinks, me.p, me.p);
        const int row = a.cu_rows ? a.cu_rows[b] : b;
        uint32_t qa[DH / 16][4];
        {
            const uint16_t* q0 = a.q + (size_t)row * a.q_ld + (size_t)(at0.j * G) * DH + 2 * tq;
#pragma unroll
            for (int ks = 0; ks < DH / 16; ++ks) {
                qa[ks][0] = g < G ? *reinterpret_cast<const uint32_t*>(q0 + (size_t)g * DH + ks * 16) : 0u;
                qa[ks][1] = g + 8 < G ? *reinterpret_cast<const uint32_t*>(q0 + (size_t)(g + 8) * DH + ks * 16) : 0u;
                qa[ks][2] = g < G ? *reinterpret_cast<const uint32_t*>(q0 + (size_t)g * DH + ks * 16 + 8) : 0u;
                qa[ks][3] = g + 8 < G ? *reinterpret_cast<const uint32_t*>(q0 + (size_t)(g + 8) * DH + ks * 16 + 8) : 0u;
            }
        }
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

        // the first unit from x_seg on that is this warp's
        int x = x_seg + ((warp - (x_seg - c0)) & (kFWarps - 1));
        for (; x < end; x += kFWarps) {
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
                float sc[BK / 8][4];
#pragma unroll
                for (int n = 0; n < BK / 8; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
                for (int ks = 0; ks < DH / 16; ++ks)
#pragma unroll
                    for (int n = 0; n < BK / 16; ++n) {
                        uint32_t kf[4];
                        ldsm4(kf, Ks + S::at(16 * n + 8 * (mi >> 1) + lr, 2 * ks + (mi & 1)));
                        mma16<F16>(sc[2 * n], qa[ks], kf[0], kf[1]);
                        mma16<F16>(sc[2 * n + 1], qa[ks], kf[2], kf[3]);
                    }
                float mx[2] = {m[0], m[1]};
#pragma unroll
                for (int n = 0; n < BK / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[n][e] *= a.scale_log2;
                        if (!whole && !seen(8 * n + 2 * tq + (e & 1))) sc[n][e] = -INFINITY;
                        mx[e >> 1] = fmaxf(mx[e >> 1], sc[n][e]);
                    }
                float base[2], corr[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                    base[h] = mx[h] == -INFINITY ? 0.0f : mx[h];
                    corr[h] = exp2_approx(m[h] - base[h]);
                    m[h] = mx[h];
                    l[h] *= corr[h];
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[n][0] *= corr[0]; acc[n][1] *= corr[0];
                    acc[n][2] *= corr[1]; acc[n][3] *= corr[1];
                }
#pragma unroll
                for (int n = 0; n < BK / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[n][e] = exp2_approx(sc[n][e] - base[e >> 1]);
                        l[e >> 1] += sc[n][e];
                    }
#pragma unroll
                for (int ks = 0; ks < BK / 16; ++ks) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float* w = sc[2 * ks + (u >> 1)] + 2 * (u & 1);
                        hi[u] = pack16<F16>(w[0], w[1]);
                        lo[u] = pack16<F16>(w[0] - unpack16<F16>((uint16_t)hi[u]), w[1] - unpack16<F16>((uint16_t)(hi[u] >> 16)));
                    }
#pragma unroll
                    for (int n = 0; n < DH / 16; ++n) {
                        uint32_t vf[4];
                        ldsm4_t(vf, Vs + S::at(16 * ks + 8 * (mi & 1) + lr, 2 * n + (mi >> 1)));
                        mma16<F16>(acc[2 * n], hi, vf[0], vf[1]);
                        mma16<F16>(acc[2 * n + 1], hi, vf[2], vf[3]);
                        mma16<F16>(acc[2 * n], lo, vf[0], vf[1]);
                        mma16<F16>(acc[2 * n + 1], lo, vf[2], vf[3]);
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
        // ---- the four warps' parts of this (session, KV head) ----
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            const int r = g + 8 * h;
            if (r < G) {
                float* rec = comb + ((size_t)warp * G + r) * DH;
                if (l[h] != 0.0f)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        *reinterpret_cast<float2*>(rec + 8 * n + 2 * tq) = make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
                if (tq == 0) {
                    float* ml = comb + (size_t)kFWarps * G * DH + ((size_t)warp * G + r) * 2;
                    ml[0] = m[h];
                    ml[1] = l[h];
                }
            }
        }
        __syncthreads();
        const bool shared_seg = s0 < c0 || s1 > c1;
        const int rec_floats = (G * (DH + 2) + 3) & ~3;   // 16-byte aligned records
        float* rec = a.partial + (size_t)(2 * blockIdx.x + (s0 <= c0 ? 0 : 1)) * rec_floats;
        const float* ml = comb + (size_t)kFWarps * G * DH;
        auto out_at = [&](int r, int d) { return a.out + (size_t)row * a.out_ld + (size_t)(at0.j * G + r) * DH + d; };
        for (int i = tid; i < G * (DH / 4); i += kFThreads) {
            const int r = i / (DH / 4), d = 4 * (i % (DH / 4));
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kFWarps; ++w) top = fmaxf(top, ml[(w * G + r) * 2]);
            const float base = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kFWarps; ++w) {
                const float lw = ml[(w * G + r) * 2 + 1];
                if (lw == 0.0f) continue;
                const float f = exp2_approx(ml[(w * G + r) * 2] - base);
                const float4 y = *reinterpret_cast<const float4*>(comb + ((size_t)w * G + r) * DH + d);
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
                // a contributor's record: its first range's if the segment began at or before the range
                auto rec_of = [&](int k) {
                    const int cta = f + k;
                    return a.partial + (size_t)(2 * cta + (s0 <= range_start(cta) ? 0 : 1)) * rec_floats;
                };
                for (int i = tid; i < n * G; i += kFThreads) {
                    const float2 y = __ldcg(reinterpret_cast<const float2*>(rec_of(i / G) + G * DH + 2 * (i % G)));
                    wts[i] = y.y == 0.0f ? -INFINITY : y.x;
                }
                __syncthreads();
                for (int r = tid; r < G; r += kFThreads) {
                    float top = -INFINITY;
                    for (int k = 0; k < n; ++k) top = fmaxf(top, wts[k * G + r]);
                    wts[n * G + r] = top == -INFINITY ? 0.0f : top;
                }
                __syncthreads();
                for (int i = tid; i < G * (DH / 4); i += kFThreads) {
                    const int r = i / (DH / 4), d = 4 * (i % (DH / 4));
                    const float base = wts[n * G + r];
                    float sum = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
                    for (int k = 0; k < n; ++k) {
                        const float* p = rec_of(k);
                        const float lk = __ldcg(p + G * DH + 2 * r + 1);
                        const float4 y = __ldcg(reinterpret_cast<const float4*>(p + r * DH + d));
                        const float w = exp2_approx(wts[k * G + r] - base);
                        if (lk == 0.0f) continue;   // a part without a key that is seen
                        sum = fmaf(lk, w, sum);
                        v[0] = fmaf(y.x, w, v[0]); v[1] = fmaf(y.y, w, v[1]);
                        v[2] = fmaf(y.z, w, v[2]); v[3] = fmaf(y.w, w, v[3]);
                    }
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                    *reinterpret_cast<uint2*>(out_at(r, d)) =
                        make_uint2(pack16<F16>(v[0] * inv, v[1] * inv), pack16<F16>(v[2] * inv, v[3] * inv));
                }
            }
        }
        __syncthreads();
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
    auto kern = paged_frame_kernel<DH, F16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L.total);
    if (e != cudaSuccess) return e;
    kern<<<grid, kFThreads, L.total, s>>>(mk, mv, a, L);
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
