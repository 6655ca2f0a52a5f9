// paged_dev.cuh -- device helpers of the paged attention kernels.
#pragma once
#include "common.cuh"
#include "paged.cuh"

namespace vc {

VC_DEV void cp_async16(void* dst_smem, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst_smem)), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}
VC_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
VC_DEV void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

VC_DEV void ldsm4(uint32_t (&r)[4], const void* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p)));
}
VC_DEV void ldsm4_t(uint32_t (&r)[4], const void* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p)));
}

template <bool F16>
VC_DEV void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16) mma_f16(d, a, b0, b1);
    else mma_bf16(d, a, b0, b1);
}

// two fp32 values as a pair of 16-bit ones (lo in the low half), each rounded once to nearest even
template <bool F16>
VC_DEV uint32_t pack16(float lo, float hi) {
    if constexpr (F16) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}
// two results as they are stored: the cache's type, or (widen, a bf16 cache) bf16 values in fp16's format
template <bool F16>
VC_DEV uint32_t pack_out(int widen, float lo, float hi) {
    const uint32_t v = pack16<F16>(lo, hi);
    if (F16 || !widen) return v;
    return pack16<true>(bf16_bits_to_f((uint16_t)v), bf16_bits_to_f((uint16_t)(v >> 16)));
}
template <bool F16>
VC_DEV float unpack16(uint16_t u) {
    if constexpr (F16) return __half2float(*reinterpret_cast<const __half*>(&u));
    else return bf16_bits_to_f(u);
}
template <bool F16>
VC_DEV constexpr uint32_t exponent_mask() { return F16 ? 0x7C00u : 0x7F80u; }
// whether either half of a pair of 16-bit values is an infinity or NaN
template <bool F16>
VC_DEV bool nonfinite2(uint32_t u) {
    constexpr uint32_t m = exponent_mask<F16>();
    return (u & m) == m || ((u >> 16) & m) == m;
}

// whether the lower 16 bits are an infinity or NaN
template <bool F16>
VC_DEV bool nonfinite1(uint32_t u) { return (u & exponent_mask<F16>()) == exponent_mask<F16>(); }

// whether one of eight 16-bit values is an infinity or NaN: the exponent's carry reaches the sign bit of its half
template <bool F16>
VC_DEV bool any_nonfinite(const uint4& x) {
    constexpr uint32_t one = F16 ? 0x04000400u : 0x00800080u, rest = 0x7FFF7FFFu;
    return ((((x.x & rest) + one) | ((x.y & rest) + one) | ((x.z & rest) + one) | ((x.w & rest) + one)) & 0x80008000u) != 0;
}
// the pair with 0 in the place of each
template <bool F16>
VC_DEV uint32_t finite2(uint32_t u) {
    constexpr uint32_t m = exponent_mask<F16>();
    return ((u & m) == m ? 0u : u & 0xffffu) | (((u >> 16) & m) == m ? 0u : u & 0xffff0000u);
}

// A wait for an mbarrier's phase of at most `limit` polls, without a branch that the compiler sees; 1: it came.  A poll
// sleeps until the phase completes or up to 10 us: a waiting warp leaves the issue slots to the others.
static constexpr uint32_t kPollLimit = 1u << 18;
VC_DEV uint32_t mbar_poll(uint64_t* bar, uint32_t parity, uint32_t limit) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n .reg .u32 i;\n mov.u32 i, %3;\n mov.u32 %0, 0;\n"
        "again:\n setp.eq.u32 p, i, 0;\n @p bra over;\n sub.u32 i, i, 1;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 10000;\n @!p bra again;\n mov.u32 %0, 1;\n"
        "over:\n}\n"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity), "r"(limit)
        : "memory");
    return done;
}

VC_DEV void tma_prefetch_map(const void* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

VC_DEV float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// the page of column `col` of session s, or -1 where it has none (or a bad one)
VC_DEV int page_of(const PagedKv& c, int s, int col) {
    const int e = c.table[(size_t)s * c.columns + col];
    return (unsigned)e < (unsigned)c.pages ? e : -1;
}

// one session of an attention call
struct AttnSession {
    int s;      // its index in the cache
    int row0;   // its first row
    int n;      // its rows
    int p0;     // the first row's position
};

VC_DEV int session_rows(const PagedAttnArgs& a, int i) {
    if (!a.cu_rows) return 1;
    const int n = a.cu_rows[i + 1] - a.cu_rows[i];
    return n < 0 ? 0 : min(n, a.rows);
}

// fills in session i; false where it is skipped (VC_DEV_INVALID where the caller's indices do not fit)
VC_DEV bool attn_session(const PagedAttnArgs& a, int i, AttnSession& o) {
    o.s = a.seqs ? a.seqs[i] : i;
    o.row0 = a.cu_rows ? a.cu_rows[i] : i;
    const int end = a.cu_rows ? a.cu_rows[i + 1] : i + 1;
    o.p0 = a.pos[i];
    const bool known = (unsigned)o.s < (unsigned)a.c.seqs;
    const int len = min(a.c.len[known ? o.s : 0], a.c.columns << a.c.page_shift);   // read along with the others
    o.n = end - o.row0;
    if (o.n == 0 || o.p0 < 0) return false;
    const bool ok = known && o.row0 >= 0 && end <= a.rows && o.n > 0 && o.p0 <= len - o.n;
    if (!ok) atomicOr(a.c.status, VC_DEV_INVALID);
    return ok;
}

// the key blocks of BK positions that queries at positions p_lo..p_hi can see: those of the sinks, then those
// from the window's start on
struct KeyBlocks {
    int n_sink, start, total;
    VC_DEV int block(int i) const { return i < n_sink ? i : start + (i - n_sink); }
};
template <int BK>
VC_DEV KeyBlocks key_blocks(int window, int sinks, int p_lo, int p_hi) {
    KeyBlocks k{0, 0, 0};
    const int end = p_hi / BK + 1;
    if (window > 0) {
        k.n_sink = (min(sinks, p_hi + 1) + BK - 1) / BK;
        k.start = max(p_lo - window + 1, 0) / BK;   // p_lo, window >= 0: no overflow
        if (k.start < k.n_sink) k.start = k.n_sink;
    }
    k.total = k.n_sink + max(end - k.start, 0);
    return k;
}

// What products cannot tell of values that are not finite (0 inf, inf - inf and a weight that is 0 in 32 bits make NaN): the
// sum of the infinities and NaN among four dimensions, d .. d + 3, of the values that the row at position p sees; 0 where
// there are none.
template <int DH>
struct SeenValues {
    const uint16_t* v;   // the layer's values, those of the KV head from here on
    const int* row;      // the session's row of the table
    int pages, page_shift, Hk, p, window, sinks;
};
template <int DH>
VC_DEV SeenValues<DH> seen_values(const PagedKv& c, int s, int j, int p) {
    return {c.v + (size_t)j * c.page * DH, c.table + (size_t)s * c.columns, c.pages, c.page_shift, c.Hk, p, c.window, c.sinks};
}
template <int DH, bool F16>
VC_DEV float4 odd_values(const SeenValues<DH> c, int d) {
    float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int t0 = 0; t0 <= c.p; t0 += 16) {   // 16 keys of a page
        if (c.window != 0 && t0 >= c.sinks && t0 + 15 <= c.p - c.window) {   // the window has given them up, and those to its start
            t0 = (c.p - c.window + 1) / 16 * 16 - 16;
            continue;
        }
        const int e = c.row[t0 >> c.page_shift];
        if ((unsigned)e >= (unsigned)c.pages) continue;
        const uint16_t* from = c.v + (((size_t)e * c.Hk << c.page_shift) + (t0 & ((1 << c.page_shift) - 1))) * DH + d;
        uint2 x[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) x[u] = __ldcg(reinterpret_cast<const uint2*>(from + u * DH));
#pragma unroll
        for (int u = 0; u < 16; ++u) {
            const int t = t0 + u;
            if (t > c.p || (c.window != 0 && t >= c.sinks && t <= c.p - c.window)) continue;
            if (nonfinite1<F16>(x[u].x)) z.x += unpack16<F16>((uint16_t)x[u].x);
            if (nonfinite1<F16>(x[u].x >> 16)) z.y += unpack16<F16>((uint16_t)(x[u].x >> 16));
            if (nonfinite1<F16>(x[u].y)) z.z += unpack16<F16>((uint16_t)x[u].y);
            if (nonfinite1<F16>(x[u].y >> 16)) z.w += unpack16<F16>((uint16_t)(x[u].y >> 16));
        }
    }
    return z;
}
// a call of its own where its registers are not to be the products' (not behind setmaxnreg: too few there for a call)
template <int DH, bool F16>
__device__ __noinline__ float4 odd_values_call(const SeenValues<DH> c, int d) { return odd_values<DH, F16>(c, d); }
// whether one of a thread's four results is not finite
VC_DEV bool odd_results(const float (&v)[4]) { return !(v[0] * 0.0f + v[1] * 0.0f + v[2] * 0.0f + v[3] * 0.0f == 0.0f); }
// ... and those that a seen infinity or NaN decides, put right (the sum of the weights is a number)
VC_DEV void decide_odd(float (&v)[4], const float4& z) {
    if (z.x != 0.0f) v[0] = z.x;
    if (z.y != 0.0f) v[1] = z.y;
    if (z.z != 0.0f) v[2] = z.z;
    if (z.w != 0.0f) v[3] = z.w;
}

// how many tiles the sessions' rows make (a whole warp calls): at most `most`, as the launch counted them from the rows
// and sessions (more only where cu_rows overlap; those sessions are refused)
VC_DEV int count_tiles(const PagedAttnArgs& a, int group, int tile_rows, int most) {
    long long n = 0;
    for (int b = threadIdx.x & 31; b < a.batch; b += 32) n += ((long long)session_rows(a, b) * group + tile_rows - 1) / tile_rows;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return (int)min(n, (long long)most);
}

// units of work (a tile and a KV head) of which a launch has fewer than CTAs: how many CTAs each gets at most ...
static constexpr int kMostSplits = 64;
VC_DEV int unit_splits(int units, int ctas) { return max(min(ctas / max(units, 1), kMostSplits), 1); }
// ... and into how many ranges its key blocks are split: two blocks or more in each (a record and its join take as long)
VC_DEV int key_splits(int blocks, int splits) { return max(min(splits, blocks / 2), 1); }

template <int N>
struct Count {
    static constexpr int value = N;
};

// a CTA's record of a unit is written: whether it was the last of `of` (all threads call)
VC_DEV bool last_to_arrive(int* counter, int of) {
    __shared__ int last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        last = atomicAdd(counter, 1) == of - 1;
        if (last) *counter = 0;
    }
    __syncthreads();
    __threadfence();
    return last != 0;
}

// Joins, in split order, the records of a unit whose key blocks were split into `of` ranges: rows first .. first + rows - 1
// of the tile, by all THREADS threads of the CTA.  A record: sums [rec_rows][DH], maxima and sums of weights [rec_rows],
// each under its own maximum; out(r): where row first + r goes, odd(r, d): odd_values of what it sees; factor: room for
// [of][rows].
template <int DH, bool F16, int THREADS, class Out, class Odd>
VC_DEV void join_records(const PagedAttnArgs& a, const float* all, int rec_rows, int of, int first, int rows, float* factor, Out out,
                         Odd odd) {
    const int tid = threadIdx.x, rec = rec_rows * (DH + 2);
    const float* tops = all + rec_rows * DH + first;   // a split that saw nothing: maximum -inf, factor 0, sums 0
    if (of <= 4) {   // a thread a row
        for (int q = tid; q < rows; q += THREADS) {
            float t[4], l[4], top = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int sp = 0; sp < 4; ++sp) {
                t[sp] = sp < of ? __ldcg(tops + (size_t)sp * rec + q) : -INFINITY;
                l[sp] = sp < of ? __ldcg(tops + (size_t)sp * rec + rec_rows + q) : 0.0f;
            }
#pragma unroll
            for (int sp = 0; sp < 4; ++sp) top = fmaxf(top, t[sp]);
            if (top == -INFINITY) top = 0.0f;
#pragma unroll
            for (int sp = 0; sp < 4; ++sp) {
                t[sp] = exp2_approx(t[sp] - top);
                sum = fmaf(l[sp], t[sp], sum);
            }
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int sp = 0; sp < 4; ++sp)
                if (sp < of) factor[sp * rows + q] = t[sp] * inv;
        }
    } else {   // eight threads a row
        for (int q = tid / 8; q < rows; q += THREADS / 8) {
            const unsigned lanes = 0xffu << (tid & 24);
            float top = -INFINITY, sum = 0.0f;
            for (int sp = tid % 8; sp < of; sp += 8) {
                factor[sp * rows + q] = __ldcg(tops + (size_t)sp * rec + q);
                top = fmaxf(top, factor[sp * rows + q]);
            }
#pragma unroll
            for (int m = 1; m < 8; m <<= 1) top = fmaxf(top, __shfl_xor_sync(lanes, top, m));
            if (top == -INFINITY) top = 0.0f;
            for (int sp = tid % 8; sp < of; sp += 8) {
                factor[sp * rows + q] = exp2_approx(factor[sp * rows + q] - top);
                sum = fmaf(__ldcg(tops + (size_t)sp * rec + rec_rows + q), factor[sp * rows + q], sum);
            }
#pragma unroll
            for (int m = 1; m < 8; m <<= 1) sum += __shfl_xor_sync(lanes, sum, m);
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            for (int sp = tid % 8; sp < of; sp += 8) factor[sp * rows + q] *= inv;
        }
    }
    __syncthreads();
    // few ranges: four pieces of a row a thread at a time; many: one, and eight ranges of it (what counts is loads in flight)
    const int total = rows * (DH / 4);
    auto gather = [&](auto pieces, auto ranges) {
        constexpr int U = decltype(pieces)::value, N = decltype(ranges)::value;
        for (int base = tid; base < total; base += U * THREADS) {
            float4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll N
            for (int sp = 0; sp < of; ++sp) {
                const float4* from = reinterpret_cast<const float4*>(all + (size_t)sp * rec + first * DH);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int idx = min(base + u * THREADS, total - 1);
                    const float f = factor[sp * rows + idx / (DH / 4)];
                    const float4 x = __ldcg(from + idx);
                    v[u].x = fmaf(x.x, f, v[u].x); v[u].y = fmaf(x.y, f, v[u].y);
                    v[u].z = fmaf(x.z, f, v[u].z); v[u].w = fmaf(x.w, f, v[u].w);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int idx = base + u * THREADS;
                if (idx >= total) continue;
                float y[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
                if (odd_results(y) && factor[idx / (DH / 4)] == factor[idx / (DH / 4)])   // (factors are NaN where the sum is)
                    decide_odd(y, odd(idx / (DH / 4), 4 * (idx % (DH / 4))));
                *reinterpret_cast<uint2*>(out(idx / (DH / 4)) + 4 * (idx % (DH / 4))) =
                    make_uint2(pack_out<F16>(a.widen, y[0], y[1]), pack_out<F16>(a.widen, y[2], y[3]));
            }
        }
    };
    if (of <= 4) gather(Count<4>{}, Count<2>{});
    else gather(Count<1>{}, Count<8>{});
}

// the session and the tile within it of the launch's `tile`-th tile; false behind the last (a whole warp calls)
VC_DEV bool find_tile(const PagedAttnArgs& a, int group, int tile_rows, int tile, int& session, int& t) {
    const int lane = threadIdx.x & 31;
    long long before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int b = b0 + lane;
        const long long mine = b < a.batch ? ((long long)session_rows(a, b) * group + tile_rows - 1) / tile_rows : 0;
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + incl > tile);
        if (hit) {
            const int l = __ffs(hit) - 1;
            session = b0 + l;
            t = (int)(tile - (before + __shfl_sync(0xffffffffu, incl - mine, l)));
            return true;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
}

}  // namespace vc
