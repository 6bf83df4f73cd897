// k4_q4_rows.cu -- K4: quantising rows of keys and values into the 4-bit cache,
// and reading them back.
//
// Both directions move each byte once and are bound by HBM: a row of D values
// is 2 D bytes in bf16 and D/2 + D/32 in the cache.  A warp owns a block of
// consecutive tokens of one head of K or of V: its rows lie next to each other
// in the cache, so the codes of the block are one contiguous run and the scale
// bytes another.  D/8 lanes hold a row, 8 values each; a group of 32 is four
// lanes, whose largest magnitude takes two shuffles.  All the warp's loads are
// issued before any arithmetic: kU rows per lane group.
#include <algorithm>
#include <atomic>

#include "q4_device.cuh"

namespace qa {

// The block of tokens, head and tensor of a warp.
struct Q4Task {
    int z, kv, h, tok0, n;  // launched sequence, K/V, head, first token, tokens (0: none)
};

template <int D, int kU>
__device__ __forceinline__ Q4Task q4_task(const Q4RowsParams &p) {
    const uint32_t w = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;  // below 2^32 (q4_rows_grid)
    Q4Task t{0, 0, 0, 0, 0};
    const uint32_t Hkv = p.Hkv, per = Hkv * p.kv_count;
    const int blk = w / per;
    if (blk >= p.nblocks) return t;
    const uint32_t r = w - blk * per;
    t.kv = p.kv_first + (r >= Hkv);
    t.h = r >= Hkv ? r - Hkv : r;
    int lo = 0, hi = p.nseq;  // block0[lo] <= blk < block0[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.block0[mid] <= blk) lo = mid; else hi = mid;
    }
    t.z = lo;
    t.tok0 = (blk - p.block0[lo]) * q4_block_tokens(D, kU);
    t.n = min(q4_block_tokens(D, kU), p.ntok[lo] - t.tok0);
    return t;
}

template <int D, int kU, bool kHeld>
__global__ void __launch_bounds__(256) q4_quantise_kernel(const __grid_constant__ Q4RowsParams p) {
    constexpr int LPR = D / 8;  // lanes per row
    constexpr int GR = D / kQ4Group;
    const unsigned FULL = 0xffffffffu;
    const Q4Task t = q4_task<D, kU>(p);
    if (t.n <= 0) return;
    const int lane = threadIdx.x & 31, sub = lane % LPR, half = lane / LPR;
    const __nv_bfloat16 *src = p.src[t.kv] + p.src_off[t.z] + t.h * p.src_head;
    uint4 x[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int i = half * kU + u;
        x[u] = make_uint4(0, 0, 0, 0);
        if (i < t.n)
            x[u] = *(reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(t.tok0 + i) * p.src_tok) + sub);
    }
    const int64_t row = static_cast<int64_t>(p.seq0 + t.z) * p.row_seq + t.h * p.row_head +
                        p.start[t.z] + t.tok0;
    uint32_t *codes = reinterpret_cast<uint32_t *>(p.codes[t.kv]) + row * (D / 8);
    uint8_t *scales = p.scales[t.kv] + row * GR;
    uint32_t mine = 0;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        if (u >= t.n) break;  // no lane group has a row u
        const int i = half * kU + u;
        uint32_t byte;
        uint4 held;
        const uint32_t w = q4_quantise8<kHeld>(x[u], byte, held);
        // The row's scale bytes gathered in one word, kept by lane u of the row's lanes.
        uint32_t s = byte << (8 * (sub / 4));
        s |= __shfl_xor_sync(FULL, s, 4);
        if (GR == 4) s |= __shfl_xor_sync(FULL, s, 8);
        if (sub == u) mine = s;
        if (i < t.n) {
            codes[static_cast<int64_t>(i) * LPR + sub] = w;
            if (kHeld)
                *(reinterpret_cast<uint4 *>(p.dst[t.kv] + p.dst_off[t.z] + t.h * p.dst_head +
                                            static_cast<int64_t>(t.tok0 + i) * p.dst_tok) + sub) = held;
        }
    }
    const int i = half * kU + sub;
    if (sub < kU && i < t.n) {
        if (GR == 4) reinterpret_cast<uint32_t *>(scales)[i] = mine;
        else reinterpret_cast<uint16_t *>(scales)[i] = static_cast<uint16_t>(mine);
    }
}

template <int D, int kU>
__global__ void __launch_bounds__(256) q4_dequantise_kernel(const __grid_constant__ Q4RowsParams p) {
    constexpr int LPR = D / 8;
    constexpr int GR = D / kQ4Group;
    // In a prefill it runs beside the kernel of the new rows, which touches none
    // of these, and the attention kernel after it sets up beside both.  That one
    // waits for this grid, whose last block is not done before the new rows are.
    if (p.beside) {
        griddep_launch_dependents();
        if (blockIdx.x == gridDim.x - 1) griddep_wait();
    }
    const Q4Task t = q4_task<D, kU>(p);
    if (t.n <= 0) return;
    const int lane = threadIdx.x & 31, sub = lane % LPR, half = lane / LPR;
    const int64_t row = static_cast<int64_t>(p.seq0 + t.z) * p.row_seq + t.h * p.row_head +
                        p.start[t.z] + t.tok0;
    const uint32_t *codes = reinterpret_cast<const uint32_t *>(p.codes[t.kv]) + row * (D / 8);
    const uint8_t *scales = p.scales[t.kv] + row * GR;
    __nv_bfloat16 *dst = p.dst[t.kv] + p.dst_off[t.z] + t.h * p.dst_head;
    const int hidden = p.hidden[t.z] - p.start[t.z] - t.tok0;  // rows of the block that nothing may see
    uint32_t w[kU], s[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int i = half * kU + u;
        w[u] = s[u] = 0;  // (a scale of zero: zeros)
        if (i < t.n && i >= hidden) {
            w[u] = codes[static_cast<int64_t>(i) * LPR + sub];
            s[u] = scales[i * GR + sub / 4];
        }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int i = half * kU + u;
        if (i < t.n)
            *(reinterpret_cast<uint4 *>(dst + static_cast<int64_t>(t.tok0 + i) * p.dst_tok) + sub) =
                q4_values8(w[u], s[u]);
    }
}

// -------------------------------------------------------------------- a prefill's rows
// RMSNorm + RoPE of the query and key rows and the quantised append of keys and
// values, in one pass: per token 2 D (Hq + 2 Hkv) bytes in, as many out (q' and
// the workspace's rows), and the codes.  Without it the workspace's rows would
// be written, read and written again.  Bound by HBM; a warp walks its share of
// the tokens with the next token's rows on the way into the other half of its
// ring (three bulk copies), as K1 does.
// RMSNorm + RoPE of this lane's 8 values of a row held by D/8 lanes; cs, sn:
// cosines and sines of its dims, the sines signed for its half.  Its sums are in the
// order of q4_norm_rope (K5): a key gets the same codes from a prefill and from a
// decode step.
template <int D>
__device__ __forceinline__ uint4 q4_transform(uint4 xv, uint4 wv, const float2 (&cs)[4],
                                              const float2 (&sn)[4], float eps) {
    constexpr int HALF = D / 16;
    const unsigned FULL = 0xffffffffu;
    const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w}, ww[4] = {wv.x, wv.y, wv.z, wv.w};
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        ss = fmaf(bf16lo(xw[e]), bf16lo(xw[e]), fmaf(bf16hi(xw[e]), bf16hi(xw[e]), ss));
#pragma unroll
    for (int o = HALF; o >= 1; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
    const float r = rsqrtf(ss * (1.0f / D) + eps);
    uint32_t y[4], partner[4], out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 h = __fmul2_rn(make_float2(bf16lo(xw[e]), bf16hi(xw[e])), make_float2(r, r));
        const uint32_t hb = pack_bf16(h.x, h.y);
        const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&hb),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&ww[e]));
        y[e] = *reinterpret_cast<const uint32_t *>(&v);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) partner[e] = __shfl_xor_sync(FULL, y[e], HALF);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 rot = __ffma2_rn(make_float2(bf16lo(partner[e]), bf16hi(partner[e])), sn[e],
                                      __fmul2_rn(make_float2(bf16lo(y[e]), bf16hi(y[e])), cs[e]));
        out[e] = pack_bf16(rot.x, rot.y);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

template <int D>
__global__ void __launch_bounds__(kQ4RowWarps * 32, 1)
    q4_prefill_rows_kernel(const __grid_constant__ Q4PrefillRowsParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, HALF = LPR / 2, GR = D / kQ4Group;
    const unsigned FULL = 0xffffffffu;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar[kQ4RowWarps * 2];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
    const K1Params &k = p.k1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane % LPR, grp = lane / LPR;
    // The next kernel (the older rows', or the attention) is a programmatic
    // dependent: it may start now and reads what this one writes only after its end.
    if (k.signal_early) griddep_launch_dependents();
    const int parts = p.parts;
    const int nq = k.Hq / parts, nkv = k.Hkv / parts;  // heads of a share
    const uint32_t qbytes = static_cast<uint32_t>(nq) * D * 2;
    const uint32_t kvbytes = static_cast<uint32_t>(nkv) * D * 2;
    const uint32_t stage_bytes = (qbytes + 2 * kvbytes + 127) & ~127u;
    uint8_t *ring = smem + static_cast<size_t>(warp) * 2 * stage_bytes;
    const uint32_t bar0 = smem_u32(&bar[2 * warp]);
    if (lane == 0) {
        mbar_init(bar0, 1);
        mbar_init(bar0 + 8, 1);
        fence_mbar_init();
    }
    __syncwarp();
    const uint4 wq = __ldg(reinterpret_cast<const uint4 *>(k.wq) + sub);
    const uint4 wk = __ldg(reinterpret_cast<const uint4 *>(k.wk) + sub);

    // Share w of the grid's warps: part w % parts of tokens w / parts, + stride, ...
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kQ4RowWarps + warp;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kQ4RowWarps / parts);
    const int part = static_cast<int>(first % parts), hq0 = part * nq, hkv0 = part * nkv;
    int64_t t = first / parts;
    auto load = [&](int64_t tok, int s) {  // lane 0 only
        const uint32_t dst = smem_u32(ring + s * stage_bytes), b = bar0 + 8 * s;
        mbar_expect_tx(b, qbytes + 2 * kvbytes);
        bulk_g2s(dst, k.q + (tok * k.Hq + hq0) * D, qbytes, b);
        bulk_g2s(dst + qbytes, k.k + (tok * k.Hkv + hkv0) * D, kvbytes, b);
        bulk_g2s(dst + qbytes + kvbytes, k.v + (tok * k.Hkv + hkv0) * D, kvbytes, b);
    };
    // Sequence and position of a token, and its (cos, sin) for this lane's dims.
    auto locate = [&](int64_t tok, int &b, int &pos, float4 (&c)[4]) {
        b = 0;
        while (b + 1 < k.nseq && tok >= k.cu[b + 1]) ++b;
        pos = k.start[b] + static_cast<int>(tok - k.cu[b]);
        const float4 *tab = reinterpret_cast<const float4 *>(
            k.rope + static_cast<int64_t>(pos < k.cap ? pos : 0) * (D / 2) + 8 * (sub % HALF));
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = __ldg(tab + e);
    };
    if (lane == 0 && t < k.T) load(t, 0);
    int b = 0, pos = 0;
    float4 tab[4];
    if (t < k.T) locate(t, b, pos, tab);
    int abort_flag = 0;  // each warp gives up on its own
    bool ok = true;
    int i = 0;
    for (; t < k.T; ++i, t += stride) {
        const int s = i & 1;
        const int64_t tn = t + stride;
        if (lane == 0 && tn < k.T) load(tn, s ^ 1);  // the warp is done with that stage
        int b_next = 0, pos_next = 0;
        float4 tab_next[4];
        if (tn < k.T) locate(tn, b_next, pos_next, tab_next);
        ok = mbar_wait(bar0 + 8 * s, (i >> 1) & 1, &abort_flag, k.err, kKernQ4Rows, 2);
        ok = __all_sync(FULL, ok);
        if (!ok) break;
        const bool in_cap = pos < k.cap;  // always, after host validation
        if (!in_cap && lane == 0) set_error(k.err, kErrBounds, kKernQ4Rows, 1);
        float2 cs[4], sn[4];
        const float sgn = sub < HALF ? -1.f : 1.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            cs[e] = make_float2(tab[e].x, tab[e].z);
            sn[e] = make_float2(sgn * tab[e].y, sgn * tab[e].w);
        }
        const uint8_t *st = ring + s * stage_bytes;
        auto staged = [&](int r) { return reinterpret_cast<const uint4 *>(st + static_cast<size_t>(r) * D * 2)[sub]; };
        constexpr int U = 4;  // independent rows per lane group at a time
#pragma unroll 1
        for (int r0 = 0; r0 < nq; r0 += RPW * U) {  // warp-uniform
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = staged(min(r0 + u * RPW + grp, nq - 1));
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = q4_transform<D>(x[u], wq, cs, sn, k.eps);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * RPW + grp;
                if (r < nq) reinterpret_cast<uint4 *>(k.qp + (t * k.Hq + hq0 + r) * D)[sub] = x[u];
            }
        }
        const int64_t ws = static_cast<int64_t>(k.seq_slot0 + b) * k.seq_stride + static_cast<int64_t>(pos) * D;
        const int64_t row = static_cast<int64_t>(p.seq0 + b) * p.row_seq + pos;
#pragma unroll 1
        for (int r0 = 0; r0 < 2 * nkv; r0 += RPW * U) {  // K rows, then V rows
            uint4 x[U], held[U];
            uint32_t codes[U], scale[U];
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = staged(nq + min(r0 + u * RPW + grp, 2 * nkv - 1));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r0 + u * RPW < nkv) {  // warp-uniform: some row of this pass is a key
                    const uint4 y = q4_transform<D>(x[u], wk, cs, sn, k.eps);
                    if (r0 + u * RPW + grp < nkv) x[u] = y;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                uint32_t byte;
                codes[u] = q4_quantise8<true>(x[u], byte, held[u]);
                scale[u] = byte << (8 * (sub / 4));
                scale[u] |= __shfl_xor_sync(FULL, scale[u], 4);
                if (GR == 4) scale[u] |= __shfl_xor_sync(FULL, scale[u], 8);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * RPW + grp;
                if (r >= 2 * nkv || !in_cap) continue;
                const int kv = r >= nkv, h = hkv0 + (kv ? r - nkv : r);
                const int64_t at = row + h * p.row_head;
                reinterpret_cast<uint4 *>((kv ? k.vc : k.kc) + ws + h * k.head_stride)[sub] = held[u];
                reinterpret_cast<uint32_t *>(p.codes[kv])[at * LPR + sub] = codes[u];
                if (sub == 0) {
                    if (GR == 4) reinterpret_cast<uint32_t *>(p.scales[kv])[at] = scale[u];
                    else reinterpret_cast<uint16_t *>(p.scales[kv])[at] = static_cast<uint16_t>(scale[u]);
                }
            }
        }
        // The warp's reads of the stage come before the next bulk copy overwrites it.
        fence_proxy_async_smem();
        __syncwarp();
        b = b_next;
        pos = pos_next;
#pragma unroll
        for (int e = 0; e < 4; ++e) tab[e] = tab_next[e];
    }
    // Given up: a copy requested for a token that was not reached lands first.
    if (lane == 0 && !ok && t + stride < k.T) {
        int dummy = 0;
        mbar_wait(bar0 + 8 * ((i + 1) & 1), ((i + 1) >> 1) & 1, &dummy, k.err, kKernQ4Rows, 3);
    }
}

bool q4_prefill_rows_fits(int Hq, int Hkv, int D) { return q4_row_parts(Hq, Hkv, D, int64_t(1) << 40, 1) > 0; }

template <int D>
static cudaError_t q4_prefill_rows_t(const Q4PrefillRowsParams &params, cudaStream_t stream) {
    static std::atomic<unsigned> configured{0u};  // devices 0..31 set up (one bit each)
    static std::atomic<int> sms_of[32] = {};
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    if (dev < 32 && ((configured.load(std::memory_order_acquire) >> dev) & 1u)) {
        sms = sms_of[dev].load(std::memory_order_relaxed);
    } else {
        cudaError_t e = cudaFuncSetAttribute(q4_prefill_rows_kernel<D>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kQ4RowSmemMost);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        if (dev < 32) {
            sms_of[dev].store(sms, std::memory_order_relaxed);
            configured.fetch_or(1u << dev, std::memory_order_release);
        }
    }
    Q4PrefillRowsParams p = params;
    p.parts = q4_row_parts(p.k1.Hq, p.k1.Hkv, D, p.k1.T, sms);
    if (p.parts < 1 || kQ4RowWarps % p.parts) return cudaErrorInvalidConfiguration;
    const int64_t need = (static_cast<int64_t>(p.k1.T) * p.parts + kQ4RowWarps - 1) / kQ4RowWarps;
    q4_prefill_rows_kernel<D><<<static_cast<unsigned>(std::min<int64_t>(need, sms)), kQ4RowWarps * 32,
                                q4_prefill_rows_smem(p.k1.Hq, p.k1.Hkv, D, p.parts), stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_q4_prefill_rows(const Q4PrefillRowsParams &p, int D, cudaStream_t stream) {
    if (p.k1.T <= 0) return cudaSuccess;
    return D == 128 ? q4_prefill_rows_t<128>(p, stream) : q4_prefill_rows_t<64>(p, stream);
}

static bool q4_rows_grid(const Q4RowsParams &p, unsigned &blocks) {
    const int64_t warps = static_cast<int64_t>(p.nblocks) * p.Hkv * p.kv_count;
    const int64_t n = (warps + 7) / 8;
    blocks = static_cast<unsigned>(n);
    return n > 0 && warps <= 0x7fffffff;
}

template <int D, int kU>
static void q4_quantise_t(const Q4RowsParams &p, unsigned blocks, cudaStream_t stream) {
    if (p.dst[0]) q4_quantise_kernel<D, kU, true><<<blocks, 256, 0, stream>>>(p);
    else q4_quantise_kernel<D, kU, false><<<blocks, 256, 0, stream>>>(p);
}

cudaError_t launch_q4_quantise(const Q4RowsParams &p, int D, cudaStream_t stream) {
    if (p.nblocks <= 0) return cudaSuccess;
    unsigned blocks;
    if (!q4_rows_grid(p, blocks)) return cudaErrorInvalidConfiguration;
    if (D == 128) {
        if (p.unroll == 8) q4_quantise_t<128, 8>(p, blocks, stream);
        else q4_quantise_t<128, 4>(p, blocks, stream);
    } else {
        if (p.unroll == 8) q4_quantise_t<64, 8>(p, blocks, stream);
        else q4_quantise_t<64, 4>(p, blocks, stream);
    }
    return cudaGetLastError();
}

cudaError_t launch_q4_dequantise(const Q4RowsParams &p, int D, cudaStream_t stream) {
    if (p.nblocks <= 0) return cudaSuccess;
    unsigned blocks;
    if (!q4_rows_grid(p, blocks) || p.unroll != 4) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.beside ? 1 : 0;
    return D == 128 ? cudaLaunchKernelEx(&cfg, q4_dequantise_kernel<128, 4>, p)
                    : cudaLaunchKernelEx(&cfg, q4_dequantise_kernel<64, 4>, p);
}

}  // namespace qa
