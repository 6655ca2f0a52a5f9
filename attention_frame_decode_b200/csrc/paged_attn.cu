// paged_attn.cu -- windowed attention over the paged KV cache: appending rows, and the attention of row
// tiles on warp-level matrix instructions.
//
// For a query at position p of session s and KV head j, with the keys t that it sees (t <= p, t < sinks or
// t > p - window, the page of t mapped):
//     o = sum_t w_t V_t / sum_t w_t,   w_t = exp2(z_t - max z),   z_t = scale log2(e) q . K_t.
// The queries of a session's rows and of the Hq / Hk heads that share KV head j are packed into one list of
// rows (row r: token r / G, head j G + r % G, G = Hq / Hk), which is cut into tiles: a KV tile that is loaded
// once serves all the heads of a group, and a window of W keys is read by a tile that spans few positions.
#include "paged_dev.cuh"

namespace vc {

// ------------------------------------------------------------------------------------------
// append: the new rows' keys and values into their pages, 16 bytes per thread.  Bound: HBM (4 Hk Dh bytes
// read and written per row).
// ------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(256) paged_append_kernel(const PagedAttnArgs a) {
    pdl_trigger();
    const int width = a.c.Hk * a.c.Dh / 8;   // 16-byte chunks per row
    const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int row = (int)(idx / width), chunk = (int)(idx % width);
    if (row >= a.rows) return;
    int i = row;
    if (a.cu_rows) {   // the last session that starts at or before the row
        int lo = 0, hi = a.batch;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.cu_rows[mid + 1] <= row) lo = mid + 1;
            else hi = mid;
        }
        i = lo;
        if (i >= a.batch) return;   // behind the last session
    }
    AttnSession o;
    if (!attn_session(a, i, o)) return;
    if (row < o.row0 || row >= o.row0 + o.n) return;
    const int t = o.p0 + row - o.row0;
    const int e = page_of(a.c, o.s, t >> a.c.page_shift);
    if (e < 0) return;
    const int j = chunk * 8 / a.c.Dh, d = chunk * 8 % a.c.Dh;
    const size_t to = (((size_t)e * a.c.Hk + j) * a.c.page + (t & (a.c.page - 1))) * a.c.Dh + d;
    *reinterpret_cast<uint4*>(a.c.k + to) = *reinterpret_cast<const uint4*>(a.kn + (size_t)row * a.k_ld + chunk * 8);
    *reinterpret_cast<uint4*>(a.c.v + to) = *reinterpret_cast<const uint4*>(a.vn + (size_t)row * a.v_ld + chunk * 8);
}

cudaError_t launch_paged_append(const PagedAttnArgs& a, cudaStream_t s) {
    const long long n = (long long)a.rows * (a.c.Hk * a.c.Dh / 8);
    paged_append_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a);
    return cudaGetLastError();
}

// ------------------------------------------------------------------------------------------
// row tiles: 64 or 128 packed rows per CTA, 16 per warp, key blocks of 64 positions double-buffered with cp.async.
// The key axis is split over `splits` CTAs where there are few tiles; the last CTA of a tile to arrive joins
// them in split order.
// ------------------------------------------------------------------------------------------
static constexpr int kTK = 64;
// 64 rows a CTA, or 128 (8 warps in place of 4)
template <int DH, int ROWS>
struct TileShape {
    static constexpr int THREADS = 2 * ROWS;
    static constexpr size_t BYTES = (size_t)(ROWS + 4 * kTK) * (DH + 8) * 2;
};

template <int DH, bool F16, int ROWS>
__global__ void __launch_bounds__(TileShape<DH, ROWS>::THREADS) paged_tile_kernel(const PagedAttnArgs a, int most_tiles, int ctas, bool join_later) {
    constexpr int kTR = ROWS, kTThreads = TileShape<DH, ROWS>::THREADS;
    constexpr int SK = DH + 8, CH = DH / 8, NT = DH / 8;
    extern __shared__ __align__(16) uint8_t smem[];
    uint16_t* Qs = reinterpret_cast<uint16_t*>(smem);   // [rows][SK]
    uint16_t* KV = Qs + kTR * SK;                         // [2 stages][K, V][64][SK]
    __shared__ uint32_t cleaned;   // chunks of 8 dimensions: infinities or NaN that some row sees were taken out of the values
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
    const int G = a.c.Hq / a.c.Hk;

    int session, tile;
    if (tid == 0) cleaned = 0;   // (barriers come before its use)
    if (blockIdx.x == 0)   // reports every session whose indices do not fit
        for (int i = tid; i < a.batch; i += kTThreads) {
            AttnSession o;
            attn_session(a, i, o);
        }
    const int tiles = count_tiles(a, G, kTR, most_tiles), units = tiles * a.c.Hk, splits = ctas ? unit_splits(units, ctas) : 1;
    const int unit = (int)blockIdx.x / splits, split = (int)blockIdx.x % splits, j = unit % a.c.Hk;
    if (unit >= units || !find_tile(a, G, kTR, tiles - 1 - unit / a.c.Hk, session, tile)) return;   // the longest rows first
    AttnSession o;
    if (!attn_session(a, session, o)) return;
    const int n_rows = o.n * G, r0 = tile * kTR;
    const int p_lo = o.p0 + r0 / G, p_hi = o.p0 + (min(r0 + kTR, n_rows) - 1) / G;
    const KeyBlocks kb = key_blocks<kTK>(a.c.window, a.c.sinks, p_lo, p_hi);
    const int of = key_splits(kb.total, splits);
    if (split >= of) return;
    const int i0 = (int)((long long)kb.total * split / of), i1 = (int)((long long)kb.total * (split + 1) / of);

    unsigned mapped_next = 0;   // of the block loaded last: 16-key groups whose page is mapped
    auto load = [&](int i) {
        mapped_next = 0;
        if (i < i1) {
            const int t0 = kb.block(i) * kTK;
            uint16_t* Ks = KV + (i & 1) * 2 * kTK * SK;
            uint16_t* Vs = Ks + kTK * SK;
            int mine = -1;   // lane u: the page of the block's u-th 16 keys
            if (lane < kTK / 16 && t0 + 16 * lane <= p_hi) mine = page_of(a.c, o.s, (t0 + 16 * lane) >> a.c.page_shift);
            mapped_next = __ballot_sync(0xffffffffu, mine >= 0);
#pragma unroll
            for (int k = 0; k < kTK * CH / kTThreads; ++k) {
                const int idx = tid + k * kTThreads, r = idx / CH, c = idx % CH, t = t0 + r;
                const int page = __shfl_sync(0xffffffffu, mine, r / 16);
                const bool in = page >= 0 && t <= p_hi;
                const size_t from = (((size_t)max(page, 0) * a.c.Hk + j) * a.c.page + (t & (a.c.page - 1))) * DH + c * 8;
                cp_async16(Ks + r * SK + c * 8, a.c.k + from, in);
                cp_async16(Vs + r * SK + c * 8, a.c.v + from, in);
            }
        }
        cp_async_commit();
    };
    for (int idx = tid; idx < kTR * CH; idx += kTThreads) {
        const int r = idx / CH, c = idx % CH, rr = r0 + r;
        const bool in = rr < n_rows;
        const size_t from = (size_t)(o.row0 + (in ? rr / G : 0)) * a.q_ld + (size_t)(j * G + (in ? rr % G : 0)) * DH + c * 8;
        cp_async16(Qs + r * SK + c * 8, a.q + from, in);
    }
    load(i0);

    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    const int pr[2] = {o.p0 + (r0 + 16 * warp + g) / G, o.p0 + (r0 + 16 * warp + g + 8) / G};
    const int mi = lane >> 3, lr = lane & 7;

    for (int i = i0; i < i1; ++i) {
        const unsigned mapped = mapped_next;
        load(i + 1);
        cp_async_wait<1>();
        __syncthreads();
        const int t0 = kb.block(i) * kTK;
        uint16_t* Ks = KV + (i & 1) * 2 * kTK * SK;
        uint16_t* Vs = Ks + kTK * SK;
        const bool whole = mapped == (1u << (kTK / 16)) - 1u && t0 + kTK - 1 <= p_lo &&
                           (a.c.window == 0 || t0 > p_hi - a.c.window || t0 + kTK - 1 < a.c.sinks);
        float s[kTK / 8][4];
#pragma unroll
        for (int n = 0; n < kTK / 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < DH / 16; ++ks) {
            uint32_t qa[4];
            ldsm4(qa, Qs + (16 * warp + 8 * (mi & 1) + lr) * SK + ks * 16 + 8 * (mi >> 1));
#pragma unroll
            for (int n = 0; n < kTK / 16; ++n) {
                uint32_t b[4];
                ldsm4(b, Ks + (16 * n + 8 * (mi >> 1) + lr) * SK + ks * 16 + 8 * (mi & 1));
                mma16<F16>(s[2 * n], qa, b[0], b[1]);
                mma16<F16>(s[2 * n + 1], qa, b[2], b[3]);
            }
        }
        auto seen = [&](int h, int key) {
            const int t = t0 + key;
            return ((mapped >> (key >> 4)) & 1u) && t <= pr[h] &&
                   (a.c.window == 0 || t < a.c.sinks || t > pr[h] - a.c.window);
        };
        float mx[2] = {m[0], m[1]};
#pragma unroll
        for (int n = 0; n < kTK / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int h = e >> 1;
                s[n][e] *= a.scale_log2;
                if (!whole && !seen(h, 8 * n + 2 * tq + (e & 1))) s[n][e] = -INFINITY;
                mx[h] = fmaxf(mx[h], s[n][e]);
            }
        float corr[2], base[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
            base[h] = mx[h] == -INFINITY ? 0.0f : mx[h];   // nothing seen so far: every weight 0
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
        for (int n = 0; n < kTK / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[n][e] = exp2_approx(s[n][e] - base[e >> 1]);
                l[e >> 1] += s[n][e];
            }
        // a value that is not finite may be under a weight of 0 for some rows and seen by others: rare, and then it is
        // taken out of the tile before the products, and the results decided by the values themselves
        if (!whole) {
            bool odd = false;
            for (int idx = tid; idx < kTK * (DH / 2); idx += kTThreads)
                odd |= nonfinite2<F16>(*reinterpret_cast<const uint32_t*>(Vs + (idx / (DH / 2)) * SK + 2 * (idx % (DH / 2))));
            if (__syncthreads_or(odd)) {
                uint32_t some = 0;   // (what no page or no later row covers is 0 already)
                for (int idx = tid; idx < kTK * DH; idx += kTThreads) {
                    uint16_t* p = Vs + (idx / DH) * SK + idx % DH;
                    if (!nonfinite1<F16>(*p)) continue;
                    *p = 0;
                    const int t = t0 + idx / DH;
                    if (a.c.window == 0 || t < a.c.sinks || t > p_lo - a.c.window) some |= 1u << (idx % DH / 8);
                }
                if (some) atomicOr(&cleaned, some);
                __syncthreads();
            }
        }
        // P in 16 bits, as the matrix instruction takes it: off by up to 2^-8 (bf16) or 2^-11 (fp16) of each weight
#pragma unroll
        for (int ks = 0; ks < kTK / 16; ++ks) {
            uint32_t pa[4];
            pa[0] = pack16<F16>(s[2 * ks][0], s[2 * ks][1]);
            pa[1] = pack16<F16>(s[2 * ks][2], s[2 * ks][3]);
            pa[2] = pack16<F16>(s[2 * ks + 1][0], s[2 * ks + 1][1]);
            pa[3] = pack16<F16>(s[2 * ks + 1][2], s[2 * ks + 1][3]);
#pragma unroll
            for (int n = 0; n < DH / 16; ++n) {
                uint32_t b[4];
                ldsm4_t(b, Vs + (16 * ks + 8 * (mi & 1) + lr) * SK + 16 * n + 8 * (mi >> 1));
                mma16<F16>(acc[2 * n], pa, b[0], b[1]);
                mma16<F16>(acc[2 * n + 1], pa, b[2], b[3]);
            }
        }
        __syncthreads();
    }
    cp_async_wait<0>();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t odd = cleaned;
#pragma unroll
        for (int n = 0; n < NT; ++n)
            if (acc[n][2 * h] * 0.0f + acc[n][2 * h + 1] * 0.0f != 0.0f) odd |= 1u << n;
        if (odd == 0 || l[h] != l[h] || r0 + 16 * warp + g + 8 * h >= n_rows) continue;
        const SeenValues<DH> values = seen_values<DH>(a.c, o.s, j, pr[h]);
#pragma unroll 1
        for (int k = 0; k < NT; ++k) {
            if (!((odd >> k) & 1u)) continue;
            const float4 z = odd_values_call<DH, F16>(values, 8 * k + 4 * (tq >> 1));
            const float z0 = tq & 1 ? z.z : z.x, z1 = tq & 1 ? z.w : z.y;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n == k && z0 != 0.0f) acc[n][2 * h] = z0;
                if (n == k && z1 != 0.0f) acc[n][2 * h + 1] = z1;
            }
        }
    }
    auto out_row = [&](int rr) { return a.out + (size_t)(o.row0 + rr / G) * a.out_ld + (size_t)(j * G + rr % G) * DH; };
    if (of == 1) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int rr = r0 + 16 * warp + g + 8 * h;
            if (rr >= n_rows) continue;
            const float inv = l[h] == 0.0f ? 0.0f : 1.0f / l[h];
            uint16_t* to = out_row(rr);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                *reinterpret_cast<uint32_t*>(to + 8 * n + 2 * tq) =
                    pack_out<F16>(a.widen, acc[n][2 * h] * inv, acc[n][2 * h + 1] * inv);
        }
        return;
    }
    // a split's record: [rows][DH] sums, then [rows] maxima and [rows] sums of weights
    constexpr int REC = kTR * (DH + 2);
    float* rec = a.partial + ((size_t)unit * splits + split) * REC;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = 16 * warp + g + 8 * h;
#pragma unroll
        for (int n = 0; n < NT; ++n)
            *reinterpret_cast<float2*>(rec + r * DH + 8 * n + 2 * tq) = make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
        if (tq == 0) {
            rec[kTR * DH + r] = m[h];
            rec[kTR * DH + kTR + r] = l[h];
        }
    }
    if (join_later || !last_to_arrive(a.merge + unit, of)) return;
    join_records<DH, F16, kTThreads>(a, a.partial + (size_t)unit * splits * REC, kTR, of, 0, min(kTR, n_rows - r0),
                                     reinterpret_cast<float*>(smem), [&](int r) { return out_row(r0 + r); },
                                     [&](int r, int d) { return odd_values_call<DH, F16>(seen_values<DH>(a.c, o.s, j, o.p0 + (r0 + r) / G), d); });
}

// ------------------------------------------------------------------------------------------
// joins as a launch of their own, 16 rows a CTA, for caches that may hold many keys: every SM reads records (by the last
// CTA of a tile to arrive, 37 records of 64 rows of 256 took 100 us).  Where there cannot be many, the last CTA to arrive
// joins: the launch takes 2 to 5 us.
// ------------------------------------------------------------------------------------------
static constexpr int kJRows = 16, kJThreads = 128;

template <int DH, bool F16, int BK>
__global__ void __launch_bounds__(kJThreads) paged_join_kernel(const PagedAttnArgs a, const JoinShape w) {
    __shared__ float factor[kMostSplits * kJRows];
    pdl_trigger();
    pdl_wait();
    const int G = a.c.Hq / a.c.Hk, unit = blockIdx.x, j = unit % a.c.Hk;
    const int tiles = count_tiles(a, G, w.tile_rows, w.most_tiles), units = tiles * a.c.Hk, splits = unit_splits(units, w.ctas);
    int session, tile;
    AttnSession o;
    if (unit >= units || !find_tile(a, G, w.tile_rows, tiles - 1 - unit / a.c.Hk, session, tile) || !attn_session(a, session, o))
        return;
    const int r0 = tile * w.tile_rows, r1 = min(r0 + w.tile_rows, o.n * G), first = blockIdx.y * kJRows;
    const int rows = min(kJRows, r1 - r0 - first);
    const KeyBlocks kb = key_blocks<BK>(a.c.window, a.c.sinks, o.p0 + r0 / G, o.p0 + (r1 - 1) / G);
    const int of = key_splits(kb.total, splits);
    if (rows <= 0 || of == 1) return;
    join_records<DH, F16, kJThreads>(a, a.partial + (size_t)unit * splits * (w.rows * (DH + 2)), w.rows, of, first, rows, factor, [&](int r) {
        const int packed = r0 + first + r;
        return a.out + (size_t)(o.row0 + packed / G) * a.out_ld + (size_t)(j * G + packed % G) * DH;
    }, [&](int r, int d) { return odd_values_call<DH, F16>(seen_values<DH>(a.c, o.s, j, o.p0 + (r0 + first + r) / G), d); });
}

template <int DH, int BK>
static cudaError_t launch_join_t(const PagedAttnArgs& a, const JoinShape& w, cudaStream_t s) {
    // units that may be split: the others are as many as half of the CTAs, or more
    const long long units = (long long)w.most_tiles * a.c.Hk, most = w.ctas / 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(units < most ? units : most), (unsigned)((w.rows + kJRows - 1) / kJRows));
    cfg.blockDim = dim3(kJThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = a.pdl;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return a.f16 ? cudaLaunchKernelEx(&cfg, paged_join_kernel<DH, true, BK>, a, w)
                 : cudaLaunchKernelEx(&cfg, paged_join_kernel<DH, false, BK>, a, w);
}

cudaError_t launch_paged_join(const PagedAttnArgs& a, const JoinShape& w, cudaStream_t s) {
    switch (a.c.Dh) {
        case 32: return launch_join_t<32, 64>(a, w, s);
        case 64: return launch_join_t<64, 64>(a, w, s);
        case 128: return w.keys == 64 ? launch_join_t<128, 64>(a, w, s) : launch_join_t<128, 128>(a, w, s);
        case 256: return launch_join_t<256, 64>(a, w, s);
    }
    return cudaErrorInvalidValue;
}

template <int DH, bool F16, int ROWS>
static cudaError_t launch_tiles_t(const PagedAttnArgs& a, cudaStream_t s) {
    using S = TileShape<DH, ROWS>;
    auto kern = paged_tile_kernel<DH, F16, ROWS>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::BYTES);
    if (e != cudaSuccess) return e;
    const long long G = a.c.Hq / a.c.Hk;
    // at most: every session's last tile may be part-filled
    const long long tiles = a.cu_rows ? (a.rows * G + ROWS - 1) / ROWS + a.batch : a.batch * ((G + ROWS - 1) / ROWS);
    const long long units = tiles * a.c.Hk;
    if (units > INT32_MAX) return cudaErrorInvalidValue;
    // the key blocks are split where that gives more SMs work: two CTAs on each, one at head dim 256
    const int ctas = a.num_sms * (DH == 256 ? 1 : 2);
    const long long least = a.cu_rows ? (a.rows * G + ROWS - 1) / ROWS : tiles;
    const bool may_split = least * a.c.Hk * 2 <= ctas, join_later = may_split && many_keys(a);
    static_assert(S::BYTES >= (size_t)kMostSplits * ROWS * 4, "room for the join's factors");
    kern<<<(unsigned)(may_split && units < ctas ? ctas : units), S::THREADS, S::BYTES, s>>>(a, (int)tiles, may_split ? ctas : 0,
                                                                                         join_later);
    e = cudaGetLastError();
    return e == cudaSuccess && join_later ? launch_paged_join(a, JoinShape{ROWS, ROWS, kTK, (int)tiles, ctas}, s) : e;
}

template <int DH, int ROWS = 64>
static cudaError_t launch_tiles(const PagedAttnArgs& a, cudaStream_t s) {
    return a.f16 ? launch_tiles_t<DH, true, ROWS>(a, s) : launch_tiles_t<DH, false, ROWS>(a, s);
}

cudaError_t launch_paged_tiles(const PagedAttnArgs& a, cudaStream_t s) {
    switch (a.c.Dh) {
        case 32: return launch_tiles<32>(a, s);
        case 64: return launch_tiles<64>(a, s);
        case 128: return launch_tiles<128>(a, s);
        case 256:
            // one CTA fills an SM's shared memory: 128 rows where the sessions have them (8 heads over 4, 16 sessions of
            // 300 rows behind 1000 positions: 318 us for 388; one of 40 rows behind 16000: 117 for 142), 64 where they
            // have not (30 rows behind 30000: 157 for 171; 4 sessions of 2 rows: 16.8 for 18.4)
            return (long long)a.rows * (a.c.Hq / a.c.Hk) > 64LL * a.batch ? launch_tiles<256, 128>(a, s) : launch_tiles<256>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace vc
